// Ownership of a paged cache's pages: reference counts, page tables.
//
// refs[p] is the number of page-table entries that name page p; a page with
// refs[p] = 0 is free.  There is no list of free pages to keep: reserve finds the
// lowest free ones in refs, fork moves the counts by what changes hands.  All of it
// is whole numbers, and no result depends on the order of atomics.
#include <cooperative_groups.h>
#include <stdint.h>

#include "cluster.cuh"
#include "cluster_size.h"
#include "internal.h"

namespace attn_skip {
namespace {

namespace cg = cooperative_groups;

constexpr int NT = 1024;  // threads a CTA of reserve
constexpr int NW = NT / 32;
constexpr int kMaxCluster = kLargeCluster;
constexpr int kChunkWords = 8;  // words of 32 pages that a warp takes at a time
constexpr int kMaxRounds = (1 << 20) / (kMaxCluster * NW * kChunkWords * 32);  // chunks of a warp

__device__ __forceinline__ int pages_of(int len, int ps) {  // ceil(len / ps), len >= 0
  return (int)(((unsigned)len + (unsigned)ps - 1u) / (unsigned)ps);
}

// Sum over the lanes below and this one's.
template <typename T>
__device__ __forceinline__ T scan_warp(T x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

__device__ __forceinline__ int sum_warp(int x) { return __reduce_add_sync(0xffffffffu, x); }

// Exclusive sum over the block's threads, and the block's total.  `tmp`: NW + 1
// values of shared memory, free again after the next barrier.
template <typename T>
__device__ __forceinline__ T scan_block(T x, T *tmp, T &total) {
  static_assert(NW <= 32, "a lane a warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T upto = scan_warp(x, lane);
  if (lane == 31) tmp[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    const T w = lane < NW ? tmp[lane] : T(0), u = scan_warp(w, lane);
    if (lane < NW) tmp[lane] = u - w;
    if (lane == 31) tmp[NW] = u;
  }
  __syncthreads();
  total = tmp[NW];
  return tmp[warp] + upto - x;
}

// Per-sequence state in shared memory.
struct Seqs {
  int *begin;      // [n + 1] requests of the sequences before (saturated at INT_MAX)
  int *first;      // [n] first entry past the cached ones; bit 30: it gets a copy of its last page
  int *page;       // [n] shared page that the sequence is about to write into, -1: none, -2: bad
  int *key;        // hash of the shared pages: page + 1 (0: none),
  int *writers;    // how many sequences write into the page,
  int *last;       // and the last of them
};
constexpr int kCopy = 1 << 30;
__host__ __device__ constexpr int hash_slots(int n) {  // a power of two, twice n where there is room
  int m = 2;
  while (m < 2 * n && m < 8192) m *= 2;
  return m;
}
__host__ __device__ constexpr size_t seq_bytes(int n) { return ((size_t)n * 12 + 4 + 15) / 16 * 16; }

// One cluster.  Every CTA works out the sequences' requests for itself and looks at its
// share of refs; the counts of free pages go round through distributed shared memory,
// after which each warp hands out its own free pages: the k-th lowest free page is the k-th
// request's, in the order of sequences, a copied page first, then the new entries.  refs,
// the table and the lengths are read before the cluster's barrier and written behind it,
// so that got_len may be kv_len.
//
// Latency bounds it: some ten steps that wait for one another, half of them barriers (64
// sequences, a pool of 20000 pages: 6.5 us; 1000 prompts, 48000 new pages of a pool of
// 262144: 11.6 us; by eight CTAs 12.5, of which 2.3 to look at refs and 2.9 to hand out).
// With a page's place among the low ones deciding who hands it out, two of eight CTAs had all
// the work (46 us); hence chunks go round the CTAs, and a word of 32 pages is handed out at a
// time, so that neighbours write to neighbours.
__global__ void __launch_bounds__(NT, 1) reserve_kernel(const __grid_constant__ ReserveArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long tmp64[NW + 1];
  const cg::cluster_group cluster = cg::this_cluster();
  cluster_started();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_seq, ps = a.page_size;
  Seqs q;
  q.begin = reinterpret_cast<int *>(smem);
  q.first = q.begin + n + 1;
  q.page = q.first + n;
  const int slots = hash_slots(n);
  q.key = reinterpret_cast<int *>(smem + seq_bytes(n));
  q.writers = q.key + slots;
  q.last = q.writers + slots;
  // Chunk c of 256 pages is that of warp c / n_cta % NW in CTA c % n_cta, so that the low
  // pages, which go first, are spread over the cluster.  A warp's chunks: rounds.
  const int all_warps = n_cta * NW, me = warp * n_cta + rank;
  uint32_t *words = reinterpret_cast<uint32_t *>(q.last + slots) + warp * a.rounds * kChunkWords;
  uint16_t *counts = reinterpret_cast<uint16_t *>(  // free pages of every chunk
      reinterpret_cast<uint32_t *>(q.last + slots) + NW * a.rounds * kChunkWords);

  // What each sequence asks for: the loads of the first ones before those of refs.
  auto last_page = [&](int s, int from, int to, int &page, int &first, int &need) {
    page = -1;
    first = need = 0;
    if (from < 0 || to < from || to > (int64_t)a.max_pages * ps) {
      page = -2;
      return;
    }
    first = pages_of(from, ps);
    need = pages_of(to, ps) - first;
    if (to > from && first * (int64_t)ps != from) {  // it writes into its last page
      page = a.table[(int64_t)s * a.max_pages + first - 1];
      if (page < 0 || page >= a.n_pages) page = -2;
    }
    if (page == -2) need = 0;
  };
  int page0 = -1, first0 = 0, need0 = 0;
  if (tid < n) last_page(tid, a.kv_len[tid], a.new_len[tid], page0, first0, need0);
  for (int i = tid; i < 3 * slots; i += NT) q.key[i] = 0;

  // The free pages of this warp's chunks.
  cluster_wait();  // (the others' shared memory is there)
#pragma unroll 4
  for (int k = 0; k < a.rounds; ++k) {
    const int c = k * all_warps + me;
    int r[kChunkWords], found = 0;
#pragma unroll
    for (int i = 0; i < kChunkWords; ++i) {
      const int p = (c * kChunkWords + i) * 32 + lane;
      r[i] = p < a.n_pages ? a.refs[p] : 1;
    }
#pragma unroll
    for (int i = 0; i < kChunkWords; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, r[i] == 0);
      if (lane == 0) words[k * kChunkWords + i] = m;
      found += __popc(m);
    }
    if (lane < n_cta) *cluster.map_shared_rank(counts + c, lane) = (uint16_t)found;
  }

  bool bad = false, shared = false;
  for (int s = tid; s < n; s += NT) {
    int page = page0, first = first0, need = need0;
    if (s != tid) last_page(s, a.kv_len[s], a.new_len[s], page, first, need);
    if (page >= 0 && a.refs[page] <= 1) page = -1;
    bad |= page == -2;
    shared |= page >= 0;
    q.begin[s] = need;
    q.first[s] = first;
    q.page[s] = page;
  }
  if (bad && rank == 0) atomicOr(a.err, kErrBadArg);
  // A sequence that writes into a shared page gets a copy of it, but for the last one
  // that holds it: where as many sequences write into a page as refs counts, the last of
  // them in the batch writes into the page itself.
  if (__syncthreads_or(shared)) {
    auto slot_of = [&](int page) {  // (there are at least as many slots as sequences)
      unsigned i = ((unsigned)page * 2654435769u) >> 15;
      while (true) {
        i &= (unsigned)slots - 1;
        const int was = atomicCAS(q.key + i, 0, page + 1);
        if (was == 0 || was == page + 1) return i;
        ++i;
      }
    };
    for (int s = tid; s < n; s += NT)
      if (q.page[s] >= 0) {
        const unsigned i = slot_of(q.page[s]);
        atomicAdd(q.writers + i, 1);
        atomicMax(q.last + i, s);
      }
    __syncthreads();
    for (int s = tid; s < n; s += NT)
      if (q.page[s] >= 0) {
        const unsigned i = slot_of(q.page[s]);
        if (q.last[i] != s || q.writers[i] < a.refs[q.page[s]]) q.first[s] |= kCopy;
      }
    __syncthreads();
  }
  // Requests of the sequences before each.  Every thread takes `per` sequences.
  {
    const int per = (n + NT - 1) / NT, s0 = min(n, tid * per), s1 = min(n, s0 + per);
    long long sum = 0, total;
    for (int s = s0; s < s1; ++s) sum += q.begin[s] + (q.first[s] >> 30);
    long long at = scan_block(sum, tmp64, total);
    for (int s = s0; s < s1; ++s) {
      const int need = q.begin[s] + (q.first[s] >> 30);
      q.begin[s] = (int)min(at, 0x7fffffffll);
      at += need;
    }
    if (tid == 0) q.begin[n] = (int)min(total, 0x7fffffffll);
  }
  cluster.sync();
  // Free pages of all chunks (every warp for itself).
  int n_free = 0;
  for (int i = lane; i < a.rounds * all_warps; i += 32) n_free += counts[i];
  n_free = sum_warp(n_free);
  // Sequences in order are served as far as the pages go (`taken` requests), and
  // those that need none and write into no shared page.
  int taken;
  {
    int lo = 0, hi = n;  // the largest i with begin[i] <= n_free, by 32 probes at a time
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
      const int c = __popc(__ballot_sync(0xffffffffu, i <= hi && q.begin[min(i, hi)] <= n_free));
      lo += c * step;
      hi = min(hi, lo + step - 1);
    }
    taken = q.begin[lo];
  }
  for (int s = rank * NT + tid; s < n; s += n_cta * NT) {
    const int page = q.page[s], upto = q.begin[s + 1];
    const int new_len = a.new_len[s];
    bool served = page != -2;
    if (upto > n_free)  // who asks for nothing (by the length: sums stop at INT_MAX)
      served = page == -1 && pages_of(new_len, ps) == q.first[s];
    const bool cow = served && (q.first[s] & kCopy);
    a.got_len[s] = served ? new_len : a.kv_len[s];
    a.copy_src[s] = cow ? page : -1;
    if (!cow) a.copy_dst[s] = -1;
    if (cow) atomicSub(a.refs + page, 1);
  }
  // This warp's free pages, a word at a time: neighbours go to neighbouring requests, most
  // often the same sequence's.
  auto owner = [&](int r, int s) {  // the largest s with begin[s] <= r, which asks for something
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (q.begin[s + 1] > r) return s;
      ++s;
    }
    int hi = n - 1;
    while (s < hi) {
      const int mid = (s + hi + 1) >> 1;
      if (q.begin[mid] <= r) s = mid;
      else hi = mid - 1;
    }
    return s;
  };
  int r0 = 0, c0 = 0, s0 = 0;  // free pages of the chunks before c0; a sequence at or before r0's
  for (int k = 0; k < a.rounds; ++k) {
    const int c = k * all_warps + me;
    int more = 0;
    for (int i = c0 + lane; i < c; i += 32) more += counts[i];
    r0 += sum_warp(more);
    if (r0 >= taken) break;
    c0 = c + 1;
    s0 = owner(r0, s0);
#pragma unroll 2
    for (int i = 0; i < kChunkWords; ++i) {
      const uint32_t m = words[k * kChunkWords + i];
      const int r = r0 + __popc(m & ((1u << lane) - 1u));
      r0 += __popc(m);
      const bool mine = (m >> lane & 1u) && r < taken;
      if (mine) {
        const int s = owner(r, s0), first = q.first[s];
        const int p = (c * kChunkWords + i) * 32 + lane;
        const int e = r - q.begin[s] - (first >> 30);  // -1: the copy
        a.refs[p] = 1;
        a.table[(int64_t)s * a.max_pages + (first & ~kCopy) + e] = p;
        if (e < 0) a.copy_dst[s] = p;
        s0 = s;
      }
      s0 = __reduce_max_sync(0xffffffffu, s0);
    }
  }
}

// ---------------------------------------------------------------------- fork --
constexpr int FT = 256;
constexpr int kEntries = 8;  // table entries a thread loads at a time
constexpr int kListed = 24;     // followers of a row that are listed
constexpr int kWindow = 4 * FT;  // pages counted at a time where there are more

// A length in range, or the nearest that is.
__device__ __forceinline__ int clip(int x, int hi, bool &bad) {
  bad |= x < 0 || x > hi;
  return min(max(x, 0), hi);
}

// One CTA a row.  Those of the new batch copy entries.  Those of the old one look through
// the parents for their followers and move each page's count by how many of these have it,
// less one for the row itself: an addition a page, however many followers there are, and
// none where one follower takes the page over.  (With every follower adding for itself, 355
// followers of one sequence of 765 pages: 28 us, 4 here.)  Latency bounds it: 512 rows of up to
// 2048 entries 6.0 us; in large batches the look through the parents, which goes with the
// square: 4096 rows of 64 entries 14 us, 65536 of four 1.0 ms.
__global__ void __launch_bounds__(FT) fork_kernel(const __grid_constant__ ForkArgs a) {
  const int tid = threadIdx.x, ps = a.page_size;
  const int most = (int)min((int64_t)a.max_pages * ps, (int64_t)0x7fffffff);
  const int n_new = a.parent ? a.n_new : 0;  // (without parents the rows stay where they are)
  bool bad = false;
  if ((int)blockIdx.x < n_new) {
    const int d = blockIdx.x, s = a.parent[d], len = a.new_len[d];
    if (s < 0 || s >= a.n_seq) {
      if ((s != -1 || len != 0) && tid == 0) atomicOr(a.err, kErrBadArg);
      return;
    }
    const int old = a.kv_len[s];
    const int32_t *from = a.table + (int64_t)s * a.max_pages;
    int32_t *to = a.out_table + (int64_t)d * a.max_pages;
    int p[kEntries];  // (entries behind the last page may be read)
    auto load = [&](int e0) {
#pragma unroll
      for (int i = 0; i < kEntries; ++i)
        p[i] = e0 + i * FT < a.max_pages ? from[e0 + i * FT] : 0;
    };
    load(tid);
    const bool lost = old < 0 || old > most;  // (the old row reports it)
    const int n = pages_of(clip(len, lost ? 0 : old, bad), ps);
    for (int e0 = tid; e0 < n; e0 += kEntries * FT) {
      if (e0 != tid) load(e0);
#pragma unroll
      for (int i = 0; i < kEntries; ++i)
        if (e0 + i * FT < n) {
          to[e0 + i * FT] = p[i];
          bad |= p[i] < 0 || p[i] >= a.n_pages;  // (counts may stay, so that nobody else looks)
        }
    }
  } else {
    const int s = blockIdx.x - n_new;
    const int old = a.kv_len[s];
    if (old < 0 || old > most) {
      if (tid == 0) atomicOr(a.err, kErrBadArg);
      return;
    }
    const int32_t *from = a.table + (int64_t)s * a.max_pages;
    const int n = pages_of(old, ps);
    // Followers, how many pages they have, and the fewest and the most.
    __shared__ int followers, fewest, largest, pages_had[kListed], had[kWindow], of_warps[FT / 32];
    int count, lo, hi;
    bool unused = false;
    if (!a.parent) {
      count = 1;
      lo = hi = pages_of(clip(a.new_len[s], old, bad), ps);
    } else {
      if (tid == 0) {
        followers = 0;
        fewest = n;
        largest = 0;
      }
      __syncthreads();
      for (int e = tid; e < n_new; e += FT)
        if (a.parent[e] == s) {
          const int pages = pages_of(clip(a.new_len[e], old, unused), ps);
          const int i = atomicAdd(&followers, 1);
          if (i < kListed) pages_had[i] = pages;
          atomicMin(&fewest, pages);
          atomicMax(&largest, pages);
        }
      __syncthreads();
      count = followers;
      lo = count ? fewest : 0;
      hi = largest;
    }
    auto add = [&](int page, int more) {
      if (page < 0 || page >= a.n_pages) bad = true;
      else if (more) atomicAdd(a.refs + page, more);
    };
    // All followers have the first `lo` pages, none those from `hi` on.
    const bool listed = count <= kListed;
    for (int e0 = (count == 1 ? lo : 0) + tid; e0 < n; e0 += kEntries * FT) {
      int p[kEntries];
#pragma unroll
      for (int i = 0; i < kEntries; ++i) p[i] = e0 + i * FT < n ? from[e0 + i * FT] : 0;
#pragma unroll
      for (int i = 0; i < kEntries; ++i) {
        const int e = e0 + i * FT;
        if (e >= n) break;
        int more = (e < lo ? count : 0) - 1;
        if (e >= lo && e < hi) {
          if (!listed) continue;
          for (int d = 0; d < count; ++d) more += pages_had[d] > e;
        }
        add(p[i], more);
      }
    }
    // Many followers: how many end at each page of a window, then sums from its end (2500 pages,
    // 8 followers 5.8 us like this, 4.2 from their list; 32: 6.0 and 6.8; 140: 5.8 and 18.5;
    // 1300: 10.4 and 142).
    for (int w = lo; !listed && w < hi; w += kWindow) {
      for (int i = tid; i < kWindow; i += FT) had[i] = 0;
      __syncthreads();
      for (int e = tid; e < n_new; e += FT)
        if (a.parent[e] == s) {
          const int pages = pages_of(clip(a.new_len[e], old, unused), ps);
          if (pages > w) atomicAdd(had + min(pages - w, kWindow) - 1, 1);
        }
      __syncthreads();
      // Thread t's four from the end, the last first.
      int sum[4], upto = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = upto += had[kWindow - 1 - 4 * tid - i];
      const int scan = scan_warp(upto, tid & 31);
      if ((tid & 31) == 31) of_warps[tid >> 5] = scan;
      __syncthreads();
      int before = scan - upto;
      for (int i = 0; i < tid >> 5; ++i) before += of_warps[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) had[kWindow - 1 - 4 * tid - i] = before + sum[i];
      __syncthreads();
      for (int i = tid; i < kWindow && w + i < hi; i += FT) add(from[w + i], had[i] - 1);
      __syncthreads();
    }
  }
  if (bad) atomicOr(a.err, kErrBadArg);
}

}  // namespace

constexpr int kMaxSeqs = 8192;

// Shared memory of a reserve by n_cta CTAs that look at refs in so many rounds.
constexpr size_t reserve_bytes(int n_seq, int rounds, int n_cta) {
  return seq_bytes(n_seq) + hash_slots(n_seq) * 3 * sizeof(int) +
         (size_t)rounds * NW * (kChunkWords * 4 + n_cta * 2);
}

size_t pages_reserve_max_seqs() { return kMaxSeqs; }
size_t pages_reserve_max_pages() { return (size_t)kMaxRounds * kMaxCluster * NW * kChunkWords * 32; }

cudaError_t launch_pages_reserve(ReserveArgs a, cudaStream_t s) {
  // A CTA alone looks at 8192 pages in one round, a cluster of eight at 65536, of sixteen at
  // 131072 (pool of 8000 pages, 16 sequences: 6.4 us by one CTA, 6.9 by eight; 20000 and 64:
  // 8.1 and 7.2; 60000 and 200: 12.9 and 9.3; by eight and by sixteen 60000 and 64: 6.4 and
  // 6.9; 70000 and 200: 9.1 and 8.7; 262144 and 64: 9.2 and 8.2).
  constexpr int kPages = NW * kChunkWords * 32;
  // The kernel's limit of shared memory is one for all threads of the program: whoever sets it
  // sets the most that a call may need, so that no call lowers it under another's launch.
  constexpr size_t most = reserve_bytes(kMaxSeqs, 2 * kMaxRounds, kPortableCluster);
  static_assert(most >= reserve_bytes(kMaxSeqs, kMaxRounds, kMaxCluster), "by sixteen too");
  auto allow = [] {
    return cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)most);
  };
  const bool large = a.n_pages > 8 * kPages;
  int n_cta = a.n_pages > kPages ? kPortableCluster : 1;
  auto rounds_by = [&](int n) { return (a.n_pages + n * kPages - 1) / (n * kPages); };
  auto bytes_by = [&](int n) { return reserve_bytes(a.n_seq, rounds_by(n), n); };
  if (large || bytes_by(n_cta) > 48 * 1024 - 1024) {  // (static shared memory counts too)
    const cudaError_t e = allow();
    if (e != cudaSuccess) return e;
  }
  if (large && large_cluster_fits((const void *)reserve_kernel, NT, bytes_by(kMaxCluster)))
    n_cta = kMaxCluster;
  a.rounds = rounds_by(n_cta);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n_cta);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes_by(n_cta);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)n_cta;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reserve_kernel, a);
}

cudaError_t launch_pages_fork(const ForkArgs &a, cudaStream_t s) {
  fork_kernel<<<(unsigned)(a.n_seq + (a.parent ? a.n_new : 0)), FT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace attn_skip
