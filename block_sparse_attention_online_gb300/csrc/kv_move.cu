// Rows and pages of the paged cache moved as they are: whole pages copied, and the
// rows that a sequence keeps moved together, in the caches of all layers at once.
#include <stdint.h>

#include "internal.h"

namespace attn_skip {
namespace {

constexpr int NT = 256;

// ---------------------------------------------------------------- whole pages --
constexpr int kVec = 4;                    // 16-byte vectors a thread
constexpr int kPiece = NT * kVec * 16;     // bytes a CTA

// One CTA: a piece of one page's k or v in one layer, or all its scales.
__global__ void __launch_bounds__(NT) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a) {
  const unsigned per_page = 2u * a.chunks + (a.kv.format != kKvBf16);
  const unsigned unit = blockIdx.x / per_page;
  unsigned c = blockIdx.x - unit * per_page;
  const unsigned layer = unit / (unsigned)a.n_pairs, i = unit - layer * (unsigned)a.n_pairs;
  const int src = a.src[i], dst = a.dst[i];
  if (src == dst) return;
  if (src < 0 || dst < 0 || src >= a.kv.n_pages || dst >= a.kv.n_pages) {
    // (an entry with -1 stands for none)
    if ((src < -1 || dst < -1 || src >= a.kv.n_pages || dst >= a.kv.n_pages) && threadIdx.x == 0)
      atomicOr(a.err, kErrBadArg);
    return;
  }
  const int rows = a.kv.Hkv * a.kv.page_size;
  const auto &l = a.kv.layer[layer];
  if (c < 2u * a.chunks) {
    const int row = a.kv.format == kKvBf16 ? 256 : a.kv.format == kKvE4m3 ? 128 : 64;
    const int64_t bytes = (int64_t)rows * row;
    const bool value = c >= (unsigned)a.chunks;
    if (value) c -= a.chunks;
    uint8_t *base = value ? l.v : l.k;
    const int64_t at = (int64_t)c * kPiece + threadIdx.x * 16;
    const uint8_t *from = base + src * a.kv.page_stride + at;
    uint8_t *to = base + dst * a.kv.page_stride + at;
    uint4 x[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (at + v * (NT * 16) < bytes) x[v] = *reinterpret_cast<const uint4 *>(from + v * (NT * 16));
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (at + v * (NT * 16) < bytes) *reinterpret_cast<uint4 *>(to + v * (NT * 16)) = x[v];
    return;
  }
  // Scale bytes (a multiple of 16: pages have at least 16 rows).
  const int n_bs = a.kv.format == kKvNvfp4 ? rows / 2 : 0;  // vectors of 16 block scales
  const int n_s = rows / 16, all = 2 * (n_s + n_bs);
  for (int v = threadIdx.x; v < all; v += NT) {
    int w = v;
    uint8_t *base;
    int64_t page;
    if (w < 2 * n_s) {
      base = w < n_s ? l.k_scale : l.v_scale;
      w = w < n_s ? w : w - n_s;
      page = rows;
    } else {
      w -= 2 * n_s;
      base = w < n_bs ? l.k_bs : l.v_bs;
      w = w < n_bs ? w : w - n_bs;
      page = (int64_t)rows * 8;
    }
    *reinterpret_cast<uint4 *>(base + dst * page + w * 16) =
        *reinterpret_cast<const uint4 *>(base + src * page + w * 16);
  }
}

// ----------------------------------------------------------------- kept rows --
// Row keep[j] of a sequence to position start + j.  One group of threads (a CTA, or a
// warp where sequences keep few rows) takes the key and value rows of one (layer,
// sequence, head), in batches: first the batch's places (position -> page, slot)
// into shared memory, then its rows, loads before stores.
//
// In place this is safe without a second buffer, because keep[j] >= start + j is
// checked: row j is read in its own batch, and what overwrites its place is row
// keep[j] - start >= j, of the same batch or a later one, stored after a barrier that
// follows the loads.
struct Place {  // as the tables say it
  int from_page, from_slot, to_page, to_slot;  // from_page < 0: nothing to move
};
constexpr Place kNowhere{-1, 0, 0, -1};  // (a slot below 0: it is no fault)

struct Move {  // of a head's row, in bytes of k and v
  int64_t from, to;  // from < 0: nothing to move
};

template <int FMT> struct RowBytes {
  static constexpr int value = FMT == kKvBf16 ? 256 : FMT == kKvE4m3 ? 128 : 64;
};

// What a group works on.
struct Unit {
  int layer, s, h;
  int n, start;              // kept rows of the sequence, position of the first
  const int32_t *keep;
  const int32_t *from, *to;  // the sequence's rows of the tables
  int from_room, to_room;    // positions that they have
};

// False where there is nothing to do (bad bounds are reported).
__device__ __forceinline__ bool unit_of(const CompactArgs &a, int layer, int s, int h, bool first,
                                        Unit &x) {
  if (layer >= a.kv.n) return false;
  const int c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
  if (c0 < 0 || c1 < c0 || c1 > a.total) {
    if (first) atomicOr(a.err, kErrBadArg);
    return false;
  }
  x.layer = layer;
  x.s = s;
  x.h = h;
  x.n = c1 - c0;
  x.start = a.start ? a.start[s] : 0;
  x.keep = a.keep + (a.per_head ? (int64_t)h * a.total : 0) + c0;
  x.from = a.table + (int64_t)s * a.max_pages;
  x.to = a.out_table ? a.out_table + (int64_t)s * a.out_max_pages : x.from;
  x.from_room = a.max_pages * a.kv.page_size;  // (at most 2^30)
  x.to_room = a.out_table ? a.out_max_pages * a.kv.page_size : x.from_room;
  return true;
}

// Where row j, of position src, comes from and goes to (from_page -1: nothing to move);
// the page ids are as they come from the tables.
__device__ __forceinline__ Place place_of(const CompactArgs &a, const Unit &x, int j, int src,
                                          bool &bad) {
  const int64_t dst = (int64_t)x.start + j;
  if (src < 0 || src >= x.from_room || dst < 0 || dst >= x.to_room || (!a.out_table && src < dst)) {
    bad = true;
    return kNowhere;
  }
  if (!a.out_table && src == dst) return kNowhere;
  const unsigned ps = (unsigned)a.kv.page_size, d = (unsigned)dst;
  const unsigned pf = a.kv.page_shift >= 0 ? (unsigned)src >> a.kv.page_shift : (unsigned)src / ps;
  const unsigned pt = a.kv.page_shift >= 0 ? d >> a.kv.page_shift : d / ps;
  return Place{x.from[pf], (int)((unsigned)src - pf * ps), x.to[pt], (int)(d - pt * ps)};
}

__device__ __forceinline__ void check_place(const CompactArgs &a, Place &r, bool &bad) {
  if (r.from_page < 0 || r.from_page >= a.kv.n_pages || r.to_page < 0 || r.to_page >= a.kv.n_pages) {
    bad |= r.to_slot >= 0;
    r.from_page = -1;
  }
}

template <int ROW>
__device__ __forceinline__ Move move_of(const CompactArgs &a, const Place &r, int head_row) {
  if (r.from_page < 0) return Move{-1, -1};
  return Move{r.from_page * a.kv.page_stride + (int64_t)(head_row + r.from_slot) * ROW,
              r.to_page * a.kv.page_stride + (int64_t)(head_row + r.to_slot) * ROW};
}

// One group of threads (a CTA, or a warp where sequences keep few rows): the key and
// value rows of one (layer, sequence, head), or a share of them.
template <int FMT, int GROUP>
__global__ void __launch_bounds__(NT) compact_kernel(const __grid_constant__ CompactArgs a) {
  constexpr int LPR = RowBytes<FMT>::value / 16;  // lanes a row
  constexpr int U = GROUP == 32 ? 2 : 4;          // rows a thread loads at a time
  constexpr int CHUNK = GROUP / LPR * U;          // rows of the group
  constexpr int BATCH = GROUP == 32 ? 32 : NT;    // rows whose places are found at once
  constexpr int GROUPS = NT / GROUP;
  static_assert(BATCH == GROUP && BATCH % CHUNK == 0, "a row a thread, whole chunks");
  __shared__ Move moves[GROUPS][BATCH];
  const int g = threadIdx.x / GROUP, t = threadIdx.x % GROUP;
  Move *at = moves[g];
  auto sync = [&] {
    if constexpr (GROUP == 32) __syncwarp();
    else __syncthreads();
  };
  unsigned i = blockIdx.x * GROUPS + g;
  auto next = [&](unsigned n) {
    const unsigned q = i / n, r = i - q * n;
    i = q;
    return (int)r;
  };
  const int split = next((unsigned)a.splits), h = next((unsigned)a.kv.Hkv), s = next((unsigned)a.n_seq);
  Unit x;
  if (!unit_of(a, (int)i, s, h, t == 0, x)) return;  // (whole groups)
  const auto &l = a.kv.layer[x.layer];
  const int head_row = h * a.kv.page_size, page_rows = a.kv.Hkv * a.kv.page_size;
  uint8_t *keys = l.k + t % LPR * 16, *values = l.v + t % LPR * 16;
  bool bad = false;
  for (int j0 = split * BATCH; j0 < x.n; j0 += a.splits * BATCH) {
    sync();  // the batch before is done with the places
    const int m = min(BATCH, x.n - j0);
    Place mine = kNowhere;
    if (t < m) mine = place_of(a, x, j0 + t, x.keep[j0 + t], bad);
    check_place(a, mine, bad);
    at[t] = move_of<RowBytes<FMT>::value>(a, mine, head_row);
    sync();
    uint8_t sc[2];
    uint2 bs[2];
    if (FMT != kKvBf16 && mine.from_page >= 0) {
      const int64_t row = (int64_t)mine.from_page * page_rows + head_row + mine.from_slot;
      sc[0] = l.k_scale[row];
      sc[1] = l.v_scale[row];
      if (FMT == kKvNvfp4) {
        bs[0] = *reinterpret_cast<const uint2 *>(l.k_bs + row * 8);
        bs[1] = *reinterpret_cast<const uint2 *>(l.v_bs + row * 8);
      }
    }
    for (int c = 0; c < m; c += CHUNK) {
      uint4 v[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t byte = at[c + t / LPR + u * (GROUP / LPR)].from;
        if (byte < 0) continue;
        v[u][0] = *reinterpret_cast<const uint4 *>(keys + byte);
        v[u][1] = *reinterpret_cast<const uint4 *>(values + byte);
      }
      sync();  // all loads up to here come before the stores below
      if (FMT != kKvBf16 && c == 0 && mine.from_page >= 0) {
        const int64_t row = (int64_t)mine.to_page * page_rows + head_row + mine.to_slot;
        l.k_scale[row] = sc[0];
        l.v_scale[row] = sc[1];
        if (FMT == kKvNvfp4) {
          *reinterpret_cast<uint2 *>(l.k_bs + row * 8) = bs[0];
          *reinterpret_cast<uint2 *>(l.v_bs + row * 8) = bs[1];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t byte = at[c + t / LPR + u * (GROUP / LPR)].to;
        if (byte < 0) continue;
        *reinterpret_cast<uint4 *>(keys + byte) = v[u][0];
        *reinterpret_cast<uint4 *>(values + byte) = v[u][1];
      }
    }
  }
  if (bad) atomicOr(a.err, kErrBadArg);
}

// In place, sequences that keep many rows: they have to go in order, so what bounds a
// (layer, sequence, head) is how much it has under way.  A CTA takes keys or values,
// and 16 * LPR bytes of each row.  Rows go chunk by chunk through a ring in shared
// memory by asynchronous copies, kStages - 1 chunks ahead of the one that is stored
// (every thread stores what it has loaded itself).  Their places are found a batch of
// rows at a time, the page ids of the batch after the next and the positions of the one
// behind it under way meanwhile.
constexpr int kStages = 4;

__device__ __forceinline__ void copy_async(uint32_t smem, const void *gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

template <int FMT, int LPR>
__global__ void __launch_bounds__(NT) compact_ring_kernel(const __grid_constant__ CompactArgs a) {
  constexpr int PARTS = RowBytes<FMT>::value / 16 / LPR;
  constexpr int U = 4;                  // rows a thread loads
  constexpr int CHUNK = NT / LPR * U;   // rows of the CTA
  constexpr int MINE = CHUNK < NT ? 2 : 4;  // places a thread finds
  constexpr int BATCH = MINE * NT, PER = BATCH / CHUNK;  // rows, chunks
  static_assert(PER >= kStages - 1, "the first loads are of the first batch, the last of the next");
  extern __shared__ __align__(16) uint4 ring[];  // [kStages][U][NT], then the places
  Move *at = reinterpret_cast<Move *>(ring + kStages * U * NT);  // [2][BATCH]
  const int t = threadIdx.x;
  unsigned i = blockIdx.x;
  auto next = [&](unsigned n) {
    const unsigned q = i / n, r = i - q * n;
    i = q;
    return (int)r;
  };
  const int part = next(PARTS), value = next(2), h = next((unsigned)a.kv.Hkv), s = next((unsigned)a.n_seq);
  Unit x;
  if (!unit_of(a, (int)i, s, h, t == 0, x)) return;
  const auto &l = a.kv.layer[x.layer];
  uint8_t *codes = (value ? l.v : l.k) + (part * LPR + t % LPR) * 16;
  uint8_t *scale = value ? l.v_scale : l.k_scale, *block = value ? l.v_bs : l.k_bs;
  const int head_row = h * a.kv.page_size, page_rows = a.kv.Hkv * a.kv.page_size;
  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  const bool with_scales = FMT != kKvBf16 && part == 0;
  bool bad = false;

  // The places of batch b, in three steps.
  auto positions = [&](int b, int (&src)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int j = b * BATCH + k * NT + t;
      src[k] = j < x.n ? x.keep[j] : -1;
    }
  };
  auto page_ids = [&](int b, const int (&src)[MINE], Place (&r)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int j = b * BATCH + k * NT + t;
      r[k] = j < x.n ? place_of(a, x, j, src[k], bad) : kNowhere;
    }
  };
  uint8_t sc[MINE];      // the scales of the batch that is in `at`,
  uint2 bs[MINE];
  int64_t sc_to[MINE];   // and the rows that they go to
  auto put = [&](int b, Place (&r)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      check_place(a, r[k], bad);
      at[(b & 1) * BATCH + k * NT + t] = move_of<RowBytes<FMT>::value>(a, r[k], head_row);
      sc_to[k] = -1;
      if (with_scales && r[k].from_page >= 0) {
        const int64_t row = (int64_t)r[k].from_page * page_rows + head_row + r[k].from_slot;
        sc[k] = scale[row];
        if (FMT == kKvNvfp4) bs[k] = *reinterpret_cast<const uint2 *>(block + row * 8);
        sc_to[k] = (int64_t)r[k].to_page * page_rows + head_row + r[k].to_slot;
      }
    }
  };
  auto load = [&](int g) {  // chunk g
    const Move *chunk = at + g * CHUNK % (2 * BATCH) + t / LPR;
    const uint32_t slot = slot0 + (g % kStages) * (U * NT * 16);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t byte = chunk[u * (NT / LPR)].from;
      if (byte >= 0) copy_async(slot + u * (NT * 16), codes + byte);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  Place ids[MINE];
  int src[MINE];
  {
    int src1[MINE];
    Place ids0[MINE];
    positions(0, src);
    positions(1, src1);
    page_ids(0, src, ids0);
    page_ids(1, src1, ids);
    positions(2, src);
    put(0, ids0);
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kStages - 1; ++g) load(g);
  for (int b = 0; b * BATCH < x.n; ++b) {
    __syncthreads();  // the batch before is done, and every thread has this one's scales
    if (with_scales) {
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        if (sc_to[k] < 0) continue;
        scale[sc_to[k]] = sc[k];
        if (FMT == kKvNvfp4) *reinterpret_cast<uint2 *>(block + sc_to[k] * 8) = bs[k];
      }
    }
    put(b + 1, ids);
    page_ids(b + 2, src, ids);
    positions(b + 3, src);
    __syncthreads();
    for (int g = b * PER; g < (b + 1) * PER && g * CHUNK < x.n; ++g) {
      load(g + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncthreads();  // every thread has chunk g
      const Move *chunk = at + g * CHUNK % (2 * BATCH) + t / LPR;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t byte = chunk[u * (NT / LPR)].to;
        if (byte >= 0)
          *reinterpret_cast<uint4 *>(codes + byte) = ring[(g % kStages) * (U * NT) + u * NT + t];
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (bad) atomicOr(a.err, kErrBadArg);
}

template <int FMT, int LPR>
cudaError_t compact_ring(const CompactArgs &a, int64_t units, cudaStream_t s) {
  units *= 2 * (RowBytes<FMT>::value / 16 / LPR);
  if (units > 0x7fffffff) return cudaErrorNotYetImplemented;
  constexpr int batch = (NT / LPR * 4 < NT ? 2 : 4) * NT;
  constexpr int smem = kStages * 4 * NT * 16 + 2 * batch * (int)sizeof(Move);
  const cudaError_t e = cudaFuncSetAttribute(compact_ring_kernel<FMT, LPR>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  compact_ring_kernel<FMT, LPR><<<(unsigned)units, NT, smem, s>>>(a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t compact_fmt(CompactArgs &a, cudaStream_t s) {
  constexpr int VECS = RowBytes<FMT>::value / 16;
  const int64_t units = (int64_t)a.kv.n * a.n_seq * a.kv.Hkv;
  const int mean = a.total / a.n_seq;
  a.splits = 1;
  if (mean <= 64) {
    const int64_t grid = (units + NT / 32 - 1) / (NT / 32);
    if (grid > 0x7fffffff) return cudaErrorNotYetImplemented;
    compact_kernel<FMT, 32><<<(unsigned)grid, NT, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (a.out_table) {  // rows may be shared out where none is overwritten
    a.splits = (mean + NT - 1) / NT;
    if (units * a.splits > 0x7fffffff) return cudaErrorNotYetImplemented;
    compact_kernel<FMT, NT><<<(unsigned)(units * a.splits), NT, 0, s>>>(a);
    return cudaGetLastError();
  }
  int cut = 1;
  while (cut < 4 && units * 2 * cut < 128) cut *= 2;
  if constexpr (VECS >= 16)
    if (cut == 4) return compact_ring<FMT, VECS / 4>(a, units, s);
  if constexpr (VECS >= 8)
    if (cut >= 2) return compact_ring<FMT, VECS / 2>(a, units, s);
  return compact_ring<FMT, VECS>(a, units, s);
}

}  // namespace

cudaError_t launch_kv_copy_pages(CopyPagesArgs a, cudaStream_t s) {
  const int row = a.kv.format == kKvBf16 ? 256 : a.kv.format == kKvE4m3 ? 128 : 64;
  const int64_t bytes = (int64_t)a.kv.Hkv * a.kv.page_size * row;
  a.chunks = (int)((bytes + kPiece - 1) / kPiece);
  const int64_t grid = (2LL * a.chunks + (a.kv.format != kKvBf16)) * a.n_pairs * a.kv.n;
  if (grid > 0x7fffffff) return cudaErrorNotYetImplemented;
  copy_pages_kernel<<<(unsigned)grid, NT, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(CompactArgs a, cudaStream_t s) {
  return a.kv.format == kKvBf16   ? compact_fmt<kKvBf16>(a, s)
         : a.kv.format == kKvE4m3 ? compact_fmt<kKvE4m3>(a, s)
                                  : compact_fmt<kKvNvfp4>(a, s);
}

}  // namespace attn_skip
