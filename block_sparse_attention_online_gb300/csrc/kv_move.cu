// Rows and pages of the paged cache moved as they are: whole pages copied, and the
// rows that a sequence keeps moved together, in the caches of all layers at once.
#include <cooperative_groups.h>
#include <stdint.h>

#include "cluster.cuh"
#include "cluster_size.h"
#include "internal.h"

namespace attn_skip {
namespace {

namespace cg = cooperative_groups;

constexpr int NT = 256;

// ---------------------------------------------------------------- whole pages --
// A page of one layer has six parts: k, v, their scales and block scales, each of whole
// 16-byte vectors (a page has at least 16 rows).
//
// Large pages go in pieces of 1024 vectors.  The parts of small ones go together, by a warp
// or a CTA; there CTAs stay and share out what there is to copy: first the entries that stand
// for a copy are listed.  DRAM bounds both.
constexpr int kVec = 4;            // vectors a thread has under way
constexpr int kPiece = NT * kVec;  // vectors of a piece
constexpr int kPairs = 512;        // entries looked at at a time

struct Parts {
  int codes, scales, blocks, all;  // vectors of k (and v), of their scales, of all parts
};

__host__ __device__ __forceinline__ Parts parts_of(const KvLayers &kv) {
  const int rows = kv.Hkv * kv.page_size;
  Parts x;
  x.codes = rows * (kv.format == kKvBf16 ? 16 : kv.format == kKvE4m3 ? 8 : 4);
  x.scales = kv.format == kKvBf16 ? 0 : rows / 16;
  x.blocks = kv.format == kKvNvfp4 ? rows / 2 : 0;
  x.all = 2 * (x.codes + x.scales + x.blocks);
  return x;
}

// Vectors [from, to) of one layer's page src, all parts in a row, to page dst; `t` of GROUP
// threads.
template <int GROUP>
__device__ __forceinline__ void copy_vectors(const KvLayers &kv, const Parts &x, int layer, int2 pair,
                                             int from, int to, int t) {
  const auto &l = kv.layer[layer];
  const int64_t src = pair.x, dst = pair.y;
  for (int i0 = from + t; i0 < to; i0 += kVec * GROUP) {
    uint4 v[kVec];
    uint8_t *out[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      int i = i0 + k * GROUP;
      if (i >= to) break;
      uint8_t *base;
      int64_t stride;
      if (i < 2 * x.codes) {
        base = i < x.codes ? l.k : l.v;
        i -= i < x.codes ? 0 : x.codes;
        stride = kv.page_stride;
      } else if (i < 2 * (x.codes + x.scales)) {
        i -= 2 * x.codes;
        base = i < x.scales ? l.k_scale : l.v_scale;
        i -= i < x.scales ? 0 : x.scales;
        stride = x.scales * 16ll;
      } else {
        i -= 2 * (x.codes + x.scales);
        base = i < x.blocks ? l.k_bs : l.v_bs;
        i -= i < x.blocks ? 0 : x.blocks;
        stride = x.blocks * 16ll;
      }
      base += (int64_t)i * 16;
      out[k] = base + dst * stride;
      v[k] = *reinterpret_cast<const uint4 *>(base + src * stride);
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (i0 + k * GROUP < to) *reinterpret_cast<uint4 *>(out[k]) = v[k];
  }
}

// Lists the entries [i0, i0 + kPairs) that stand for a copy, in their order (it is the same
// in every CTA); returns how many.
__device__ __forceinline__ int list_pairs(const CopyPagesArgs &a, int i0, int2 *pairs, int *counts,
                                          bool &bad) {
  constexpr int ROUNDS = kPairs / NT, WARPS = NT / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int2 mine[ROUNDS];
  unsigned is[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int i = i0 + k * NT + t;
    mine[k].x = i < a.n_pairs ? a.src[i] : -1;
    mine[k].y = i < a.n_pairs ? a.dst[i] : -1;
  }
  __syncthreads();  // the entries before are done with
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int2 p = mine[k];
    const bool fine = p.x >= -1 && p.y >= -1 && p.x < a.kv.n_pages && p.y < a.kv.n_pages;
    bad |= !fine;
    is[k] = __ballot_sync(0xffffffffu, fine && p.x >= 0 && p.y >= 0 && p.x != p.y);
    if (lane == 0) counts[k * WARPS + warp] = __popc(is[k]);
  }
  __syncthreads();
  int n = 0, before[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS * WARPS; ++k) {
    if (k % WARPS == warp) before[k / WARPS] = n;
    n += counts[k];
  }
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k)
    if (is[k] >> lane & 1u) pairs[before[k] + __popc(is[k] & ((1u << lane) - 1u))] = mine[k];
  __syncthreads();
  return n;
}

// GROUP threads for all parts of a page in one layer.
template <int GROUP>
__global__ void __launch_bounds__(NT, 4) copy_small_kernel(const __grid_constant__ CopyPagesArgs a) {
  __shared__ int2 pairs[kPairs];
  __shared__ int counts[kPairs / 32];
  const Parts x = parts_of(a.kv);
  bool bad = false;
  for (int i0 = 0; i0 < a.n_pairs; i0 += kPairs) {
    const int n = list_pairs(a, i0, pairs, counts, bad);
    const int64_t all = (int64_t)n * a.kv.n, step = (int64_t)gridDim.x * (NT / GROUP);
    for (int64_t w = (int64_t)blockIdx.x * (NT / GROUP) + threadIdx.x / GROUP; w < all; w += step) {
      const int layer = (int)(w / n);
      copy_vectors<GROUP>(a.kv, x, layer, pairs[w - (int64_t)layer * n], 0, x.all, threadIdx.x % GROUP);
    }
  }
  if (bad) atomicOr(a.err, kErrBadArg);
}

// Large pages: a CTA for up to kTogether pieces of a page's k or v in one layer, or for all
// its scales; entries without a page cost a CTA that looks at them.  96 pages of 64 bf16 rows
// and 8 heads in 32 layers, 1.6 GB: 234 us (6.9 TB/s), 32 entries without a page among them;
// one page of 256 rows in 40 layers among 35 such entries 21 us (a CTA a piece: 55).
constexpr int kTogether = 4;

__global__ void __launch_bounds__(NT, 8) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a) {
  const Parts x = parts_of(a.kv);
  const unsigned of_codes = (unsigned)(x.codes + kTogether * kPiece - 1) / (kTogether * kPiece);
  const unsigned per_page = 2 * of_codes + (x.scales > 0);
  const unsigned page = blockIdx.x / per_page, layer = page / (unsigned)a.n_pairs;
  const unsigned c = blockIdx.x - page * per_page, i = page - layer * (unsigned)a.n_pairs;
  const int t = threadIdx.x, src = a.src[i], dst = a.dst[i];
  if (src < -1 || dst < -1 || src >= a.kv.n_pages || dst >= a.kv.n_pages) {
    if (t == 0) atomicOr(a.err, kErrBadArg);
    return;
  }
  if (src == dst || src < 0 || dst < 0) return;  // (-1 stands for none)
  const auto &l = a.kv.layer[layer];
  if (c < 2 * of_codes) {
    int64_t v0 = (int64_t)(c < of_codes ? c : c - of_codes) * (kTogether * kPiece) + t;
    uint8_t *base = c < of_codes ? l.k : l.v;
    const uint8_t *in = base + src * a.kv.page_stride;
    uint8_t *out = base + dst * a.kv.page_stride;
#pragma unroll 1
    for (int r = 0; r < kTogether; ++r, v0 += kPiece) {
      uint4 v[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (v0 + k * NT < x.codes) v[k] = *reinterpret_cast<const uint4 *>(in + (v0 + k * NT) * 16);
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (v0 + k * NT < x.codes) *reinterpret_cast<uint4 *>(out + (v0 + k * NT) * 16) = v[k];
    }
    return;
  }
  const int all = 2 * (x.scales + x.blocks);
  for (int v = t; v < all; v += NT) {
    const bool block = v >= 2 * x.scales;
    const int each = block ? x.blocks : x.scales, w = block ? v - 2 * x.scales : v;
    const bool value = w >= each;
    uint8_t *base = (block ? (value ? l.v_bs : l.k_bs) : (value ? l.v_scale : l.k_scale)) +
                    (int64_t)(value ? w - each : w) * 16;
    *reinterpret_cast<uint4 *>(base + (int64_t)dst * each * 16) =
        *reinterpret_cast<const uint4 *>(base + (int64_t)src * each * 16);
  }
}

// ----------------------------------------------------------------- kept rows --
// Row keep[j] of a sequence to position start + j, in each head, in each layer.  A row's
// place is found once (position -> page, slot -> bytes) and shared by the threads that
// move it, 16 bytes each.
//
// Into other pages any row may go at any time: CTAs take 256 rows of the batch each.  In
// place no second buffer is needed either, because keep[j] >= start + j is checked: what
// overwrites the place that row j comes from is row keep[j] - start >= j.  So a (layer,
// sequence, head) goes through its rows in chunks, the chunk's loads before its stores,
// with a barrier between them.
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

// What a group of threads works on in place, or a row's sequence.
struct Unit {
  int n, start;              // kept rows of the sequence, position of the first
  const int32_t *keep;
  const int32_t *from, *to;  // the sequence's rows of the tables
  int from_room, to_room;    // positions that they have (at most 2^30)
};

__device__ __forceinline__ bool good_bounds(const CompactArgs &a, int c0, int c1) {
  return c0 >= 0 && c1 >= c0 && c1 <= a.total;
}

// Head h of sequence s, whose rows of keep are [c0, c1).
__device__ __forceinline__ Unit unit_of(const CompactArgs &a, int s, int h, int c0, int c1) {
  Unit x;
  x.n = c1 - c0;
  x.start = a.start ? a.start[s] : 0;
  x.keep = a.keep + (a.per_head ? (int64_t)h * a.total : 0) + c0;
  x.from = a.table + (int64_t)s * a.max_pages;
  x.to = a.out_table ? a.out_table + (int64_t)s * a.out_max_pages : x.from;
  x.from_room = a.max_pages * a.kv.page_size;
  x.to_room = a.out_table ? a.out_max_pages * a.kv.page_size : x.from_room;
  return x;
}

// Remainder by n, the quotient stays.
__device__ __forceinline__ int take(unsigned &i, unsigned n) {
  const unsigned q = i / n, r = i - q * n;
  i = q;
  return (int)r;
}

// Where row j, of position src, comes from and goes to (kNowhere: nothing to move);
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

// A thread's row's scales, of keys and values.
template <int FMT> struct Scales {
  uint8_t s[2];
  uint2 b[2];
  __device__ __forceinline__ void load(const KvLayers &kv, int layer, int64_t row) {
    const auto &l = kv.layer[layer];
    s[0] = l.k_scale[row];
    s[1] = l.v_scale[row];
    if constexpr (FMT == kKvNvfp4) {
      b[0] = *reinterpret_cast<const uint2 *>(l.k_bs + row * 8);
      b[1] = *reinterpret_cast<const uint2 *>(l.v_bs + row * 8);
    }
  }
  __device__ __forceinline__ void store(const KvLayers &kv, int layer, int64_t row) const {
    const auto &l = kv.layer[layer];
    l.k_scale[row] = s[0];
    l.v_scale[row] = s[1];
    if constexpr (FMT == kKvNvfp4) {
      *reinterpret_cast<uint2 *>(l.k_bs + row * 8) = b[0];
      *reinterpret_cast<uint2 *>(l.v_bs + row * 8) = b[1];
    }
  }
};
template <> struct Scales<kKvBf16> {
  __device__ __forceinline__ void load(const KvLayers &, int, int64_t) {}
  __device__ __forceinline__ void store(const KvLayers &, int, int64_t) const {}
};

// The key and value rows of a group's threads (its `at`, one row a thread, is filled by
// all of them) move, in chunks; `mine` is this thread's own place.
template <int FMT, int GROUP, int U, typename Sync>
__device__ __forceinline__ void move_rows(const CompactArgs &a, int layer, int head_row, const Move *at,
                                          const Place &mine, int t, int m, Sync sync) {
  constexpr int LPR = RowBytes<FMT>::value / 16;  // lanes a row
  constexpr int CHUNK = GROUP / LPR * U;          // rows of the group
  static_assert(GROUP % CHUNK == 0, "whole chunks");
  const auto &l = a.kv.layer[layer];
  uint8_t *keys = l.k + t % LPR * 16, *values = l.v + t % LPR * 16;
  const int page_rows = a.kv.Hkv * a.kv.page_size;
  Scales<FMT> sc;
  if (mine.from_page >= 0)
    sc.load(a.kv, layer, (int64_t)mine.from_page * page_rows + head_row + mine.from_slot);
  for (int c = 0; c < m; c += CHUNK) {
    uint4 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t byte = at[c + t / LPR + u * (GROUP / LPR)].from;
      if (byte < 0) continue;
      v[u][0] = *reinterpret_cast<const uint4 *>(keys + byte);
      v[u][1] = *reinterpret_cast<const uint4 *>(values + byte);
    }
    sync();  // in place: all loads up to here come before the stores below
    if (c == 0 && mine.from_page >= 0)
      sc.store(a.kv, layer, (int64_t)mine.to_page * page_rows + head_row + mine.to_slot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t byte = at[c + t / LPR + u * (GROUP / LPR)].to;
      if (byte < 0) continue;
      *reinterpret_cast<uint4 *>(keys + byte) = v[u][0];
      *reinterpret_cast<uint4 *>(values + byte) = v[u][1];
    }
  }
}

// Bounds that do not ascend: a row may be of several sequences, and a search for one of them may
// find none.  The rows of every sequence with good bounds, in one (layer, head), by one CTA; what
// others move too comes out the same.
template <int FMT>
__device__ __noinline__ void compact_out_each(const CompactArgs &a, int layer, int h, Move *at) {
  const int t = threadIdx.x, head_row = h * a.kv.page_size;
  bool bad = true;
  for (int s = 0; s < a.n_seq; ++s) {
    const int c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
    if (!good_bounds(a, c0, c1)) continue;
    const Unit x = unit_of(a, s, h, c0, c1);
    for (int j0 = 0; j0 < x.n; j0 += NT) {
      Place mine = kNowhere;
      if (j0 + t < x.n) mine = place_of(a, x, j0 + t, x.keep[j0 + t], bad);
      check_place(a, mine, bad);
      __syncthreads();  // the rows before are done with the places
      at[t] = move_of<RowBytes<FMT>::value>(a, mine, head_row);
      __syncthreads();
      move_rows<FMT, NT, 4>(a, layer, head_row, at, mine, t, min(NT, x.n - j0), [] {});
    }
  }
  atomicOr(a.err, kErrBadArg);
}

// Into other pages: one CTA for 256 rows of the batch in one (layer, head), whatever
// sequences they are of, and one that looks at all bounds for it.  11000 rows of 4 heads in 4
// layers, NVFP4: 6.6 us, 5.4 for the bytes; 8196 of 8 heads in 8 layers, bf16: 83 us, 80 for
// the bytes.  (A CTA a stretch of one sequence in turn: 10 and 85 us.)
template <int FMT>
__global__ void __launch_bounds__(NT, 4) compact_out_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ Move at[NT];
  const int t = threadIdx.x;
  bool bad = false;
  unsigned i = blockIdx.x;
  const unsigned units = (unsigned)(a.kv.n * a.kv.Hkv), look = gridDim.x - units;
  if (i >= look) {
    for (int s = t; s < a.n_seq; s += NT) bad |= !good_bounds(a, a.cu_keep[s], a.cu_keep[s + 1]);
    if (!__syncthreads_or(bad)) return;
    i -= look;
    const int h = take(i, (unsigned)a.kv.Hkv);
    compact_out_each<FMT>(a, (int)i, h, at);
    return;
  }
  const int j0 = take(i, (unsigned)((a.total + NT - 1) / NT)) * NT, h = take(i, (unsigned)a.kv.Hkv);
  const int layer = (int)i, row = j0 + t;
  const int head_row = h * a.kv.page_size;
  Place mine = kNowhere;
  if (row < a.total) {
    int s = 0, hi = a.n_seq;  // entries of cu_keep[1..] at or before the row: its sequence
    while (s < hi) {
      const int mid = (s + hi) >> 1;
      if (a.cu_keep[mid + 1] <= row) s = mid + 1;
      else hi = mid;
    }
    if (s < a.n_seq) {
      const int c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
      if (good_bounds(a, c0, c1) && row >= c0 && row < c1) {
        const Unit x = unit_of(a, s, h, c0, c1);
        mine = place_of(a, x, row - c0, x.keep[row - c0], bad);
      }
    }
  }
  check_place(a, mine, bad);
  at[t] = move_of<RowBytes<FMT>::value>(a, mine, head_row);
  __syncthreads();
  move_rows<FMT, NT, 4>(a, layer, head_row, at, mine, t, min(NT, a.total - j0), [] {});
  if (bad) atomicOr(a.err, kErrBadArg);
}

// In place, sequences that keep at most a.few rows: a warp for a (layer, sequence, head).
// Latency bounds it (bounds, positions, page ids, rows: 16 sequences of up to 4 rows, 8
// heads, 32 layers, E4M3 3.4 us).
template <int FMT>
__global__ void __launch_bounds__(NT, 4) compact_warp_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ Move moves[NT / 32][32];
  const int t = threadIdx.x & 31;
  Move *at = moves[threadIdx.x >> 5];
  unsigned i = blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  const int h = take(i, (unsigned)a.kv.Hkv), s = take(i, (unsigned)a.n_seq), layer = (int)i;
  if (layer >= a.kv.n) return;
  const int c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
  if (!good_bounds(a, c0, c1)) {
    if (t == 0) atomicOr(a.err, kErrBadArg);
    return;
  }
  const Unit x = unit_of(a, s, h, c0, c1);
  if (x.n > a.few) return;  // the other kernel's
  const int head_row = h * a.kv.page_size;
  bool bad = false;
  for (int j0 = 0; j0 < x.n; j0 += 32) {
    __syncwarp();  // the rows before are done with the places
    Place mine = kNowhere;
    if (j0 + t < x.n) mine = place_of(a, x, j0 + t, x.keep[j0 + t], bad);
    check_place(a, mine, bad);
    at[t] = move_of<RowBytes<FMT>::value>(a, mine, head_row);
    __syncwarp();
    move_rows<FMT, 32, 2>(a, layer, head_row, at, mine, t, min(32, x.n - j0), [] { __syncwarp(); });
  }
  if (bad) atomicOr(a.err, kErrBadArg);
}

// Calls f(unit) for the units whose sequence keeps more than a.few rows and at most a.many,
// out of every `step`th from `first` on; 32 are looked at at a time, by every warp.
// `per_seq`: units a sequence (and layer).
template <typename F>
__device__ __forceinline__ void for_units(const CompactArgs &a, unsigned per_seq, unsigned first,
                                         unsigned step, bool &bad, F f) {
  const int64_t all = (int64_t)a.kv.n * a.n_seq * per_seq;
  for (int64_t u0 = first; u0 < all; u0 += 32ll * step) {
    const int64_t u = u0 + (int64_t)(threadIdx.x & 31) * step;
    bool is = false;
    if (u < all) {
      unsigned i = (unsigned)(u / per_seq);
      const int s = take(i, (unsigned)a.n_seq), c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
      is = good_bounds(a, c0, c1) && c1 - c0 > a.few && c1 - c0 <= a.many;
      bad |= !good_bounds(a, c0, c1);
    }
    for (unsigned many = __ballot_sync(0xffffffffu, is); many; many &= many - 1)
      f(u0 + (int64_t)(__ffs(many) - 1) * step);
  }
}

// In place, many (layer, sequence, head) of medium length: a CTA each, 256 rows at a time,
// keys and values.  Four CTAs an SM hide each other's way (bounds, positions, page ids, then
// loads and stores in turn): 1024 of 512 rows, bf16, 55 us, 52 by rings; 4096 of up to 512
// at the copy rate.
template <int FMT>
__global__ void __launch_bounds__(NT, 4) compact_cta_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ Move at[NT];
  const int t = threadIdx.x;
  bool bad = false;
  for_units(a, (unsigned)a.kv.Hkv, blockIdx.x, gridDim.x, bad, [&](int64_t unit) {
    unsigned i = (unsigned)unit;
    const int h = take(i, (unsigned)a.kv.Hkv), s = take(i, (unsigned)a.n_seq);
    const Unit x = unit_of(a, s, h, a.cu_keep[s], a.cu_keep[s + 1]);
    const int head_row = h * a.kv.page_size;
    for (int j0 = 0; j0 < x.n; j0 += NT) {
      Place mine = kNowhere;
      if (j0 + t < x.n) mine = place_of(a, x, j0 + t, x.keep[j0 + t], bad);
      check_place(a, mine, bad);
      __syncthreads();  // the rows before are done with the places
      at[t] = move_of<RowBytes<FMT>::value>(a, mine, head_row);
      __syncthreads();
      move_rows<FMT, NT, 4>(a, (int)i, head_row, at, mine, t, min(NT, x.n - j0),
                            [] { __syncthreads(); });
    }
  });
  if (bad) atomicOr(a.err, kErrBadArg);
}

// In place, sequences that keep many rows: they have to go in order, so what bounds a
// (layer, sequence, head) is how much it has under way, and at what rate an SM loads and
// stores rows.  A CTA takes keys or values; where there are few of these, the CTAs of a
// cluster share the rows out, chunk by chunk in turn, with the cluster's barrier in place of
// the CTA's.  Chunks go through a ring in shared memory by asynchronous copies, kStages - 1
// ahead of the one that is stored (every thread stores what it has loaded itself).  Their
// places are found a batch of chunks at a time, the page ids of the batch after the next
// and the positions of the one behind it under way meanwhile.  8196 rows of 8 heads in 8
// layers, bf16: 85 us, 80 for the bytes at the copy rate; with loads one chunk ahead in
// registers 110, without 244.
constexpr int kStages = 5;

__device__ __forceinline__ void copy_async(uint32_t smem, const void *gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

// The chunk and batch sizes of a CTA, and its shared memory.
template <int FMT> struct Ring {
  static constexpr int LPR = RowBytes<FMT>::value / 16;  // lanes a row
  static constexpr int U = 4;                            // rows a thread loads
  static constexpr int CHUNK = NT / LPR * U;             // rows of the CTA
  static constexpr int MINE = CHUNK < NT ? 2 : 4;        // places a thread finds
  static constexpr int BATCH = MINE * NT, PER = BATCH / CHUNK;  // rows, chunks
  static constexpr int BYTES = kStages * U * NT * 16 + 2 * BATCH * (int)sizeof(Move);
  static_assert(PER >= kStages - 1, "the first loads are of the first batch, the last of the next");
};

// One (layer, sequence, head), keys or values; the whole cluster of n_cta CTAs.
template <int FMT>
__device__ __forceinline__ void compact_unit(const CompactArgs &a, const Unit &x, int layer, int h,
                                             int value, int n_cta, int rank, uint4 *ring, bool &bad) {
  using R = Ring<FMT>;
  constexpr int LPR = R::LPR, U = R::U, CHUNK = R::CHUNK, MINE = R::MINE, BATCH = R::BATCH;
  constexpr int PER = R::PER;
  Move *at = reinterpret_cast<Move *>(ring + kStages * U * NT);  // [2][BATCH], behind [kStages][U][NT]
  const int t = threadIdx.x;
  const auto &l = a.kv.layer[layer];
  uint8_t *codes = (value ? l.v : l.k) + t % LPR * 16;
  uint8_t *scale = value ? l.v_scale : l.k_scale, *block = value ? l.v_bs : l.k_bs;
  const int head_row = h * a.kv.page_size, page_rows = a.kv.Hkv * a.kv.page_size;
  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  // The barrier orders the loads of one CTA before the stores of another.  The loads are
  // complete when their thread arrives (copies have been waited for, scales written down),
  // and the wait keeps the stores behind it, so that the cluster's barrier has nothing to
  // release: that would wait for the thread's earlier stores too, 0.6 us a chunk.  (The memory
  // model speaks of a release here; that a load whose value is in hand sees no store made after
  // it is a matter of the machine that this is written for.)
  auto sync = [&] {
    if (n_cta == 1) {
      __syncthreads();
    } else {
      cluster_started();
      cluster_wait();
    }
  };
  // The sequence's row of place k of this thread in batch b: chunk c of this CTA is chunk
  // c * n_cta + rank of the sequence.
  auto row_of = [&](int b, int k) {
    const int r = k * NT + t;
    return ((b * PER + r / CHUNK) * n_cta + rank) * CHUNK + r % CHUNK;
  };

  // The places of batch b, in three steps.
  auto positions = [&](int b, int (&src)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int j = row_of(b, k);
      src[k] = j < x.n ? x.keep[j] : -1;
    }
  };
  auto page_ids = [&](int b, const int (&src)[MINE], Place (&r)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int j = row_of(b, k);
      r[k] = j < x.n ? place_of(a, x, j, src[k], bad) : kNowhere;
    }
  };
  uint8_t sc[MINE];      // the scales of the batch that is in `at`,
  uint2 bs[MINE];
  int64_t sc_to[MINE];   // and the rows that they go to
  __shared__ volatile uint32_t loaded[FMT == kKvBf16 ? 1 : NT];
  auto put = [&](int b, Place (&r)[MINE]) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      check_place(a, r[k], bad);
      at[(b & 1) * BATCH + k * NT + t] = move_of<RowBytes<FMT>::value>(a, r[k], head_row);
      sc_to[k] = -1;
      if (FMT != kKvBf16 && r[k].from_page >= 0) {
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
  for (int b = 0; b * BATCH * n_cta < x.n; ++b) {
    if (FMT != kKvBf16) {  // (writing them down waits for the loads of the scales)
      uint32_t all = 0;
#pragma unroll
      for (int k = 0; k < MINE; ++k)
        if (sc_to[k] >= 0) all ^= FMT == kKvNvfp4 ? sc[k] ^ bs[k].x ^ bs[k].y : sc[k];
      loaded[t] = all;
    }
    sync();  // the batch before is done, and every thread has this one's scales
    if (FMT != kKvBf16) {
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
    for (int g = b * PER; g < (b + 1) * PER && g * CHUNK * n_cta < x.n; ++g) {
      load(g + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      sync();  // every thread has chunk g
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
  __syncthreads();  // the unit is done with the places
}

template <int FMT>
__global__ void __launch_bounds__(NT) compact_ring_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ __align__(16) uint4 ring[];
  const cg::cluster_group cluster = cg::this_cluster();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  bool bad = false;
  for_units(a, 2u * a.kv.Hkv, blockIdx.x / n_cta, gridDim.x / n_cta, bad, [&](int64_t unit) {
    unsigned i = (unsigned)(unit >> 1);
    const int h = take(i, (unsigned)a.kv.Hkv), s = take(i, (unsigned)a.n_seq);
    const Unit x = unit_of(a, s, h, a.cu_keep[s], a.cu_keep[s + 1]);
    compact_unit<FMT>(a, x, (int)i, h, (int)(unit & 1), n_cta, rank, ring, bad);
  });
  if (bad) atomicOr(a.err, kErrBadArg);
}

template <int FMT>
cudaError_t compact_ring(const CompactArgs &a, int64_t at_once, cudaStream_t s) {
  constexpr int smem = Ring<FMT>::BYTES;
  const cudaError_t e = cudaFuncSetAttribute(compact_ring_kernel<FMT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.kv.n * a.n_seq * a.kv.Hkv * 2;
  // CTAs a cluster, until there are 128 of them: bf16, 8196 rows of 8 heads in one layer 70 us
  // by one, 41, 22, 18 and 19.5 by two, four, eight and sixteen; of 4 heads 13.7 by eight, 11.6
  // by sixteen, of one 13.6 and 8.9; in 8 layers 85 by one, 97, 89 and 90 by two to eight.
  int n_cta = 1;
  while (n_cta < kLargeCluster && 2 * at_once * n_cta < 128) n_cta *= 2;
  if (n_cta == kLargeCluster &&
      !large_cluster_fits((const void *)compact_ring_kernel<FMT>, NT, smem))
    n_cta = kPortableCluster;
  const int64_t clusters = a.few > 0 ? min(units, (int64_t)152 * 2 / n_cta) : units;
  if (clusters * n_cta > 0x7fffffff) return cudaErrorNotYetImplemented;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * n_cta));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)n_cta;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compact_ring_kernel<FMT>, a);
}

template <int FMT>
cudaError_t compact_fmt(CompactArgs &a, cudaStream_t s) {
  const int64_t units = (int64_t)a.kv.n * a.n_seq * a.kv.Hkv;
  if (a.out_table) {
    const int64_t grid = (int64_t)a.kv.n * a.kv.Hkv * ((a.total + NT - 1) / NT + 1);
    if (grid > 0x7fffffff) return cudaErrorNotYetImplemented;
    compact_out_kernel<FMT><<<(unsigned)grid, NT, 0, s>>>(a);
    return cudaGetLastError();
  }
  // Many (layer, sequence, head) of few rows go to warps, where that is all there is to do
  // (1024 of them, 8 rows of bf16: 3.4 us by warps, 5.4 by CTAs) or saves more than the
  // launch for others (4096, up to 8 rows: 7.2 us with it, 14.5 by CTAs; up to 32: 18 and 17).
  const int mean = a.total / a.n_seq, few = 12288 / (2 * RowBytes<FMT>::value);
  const bool all_few = a.total <= 4 * few;  // (at worst one sequence has them all: 11 us)
  a.few = units >= 608 && (all_few || (units >= 2048 && mean <= few / 2)) ? few : 0;
  if (a.few > 0 && all_few) a.few = a.total;
  if (a.few > 0) {
    const int64_t grid = (units + NT / 32 - 1) / (NT / 32);
    compact_warp_kernel<FMT><<<(unsigned)grid, NT, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.total <= a.few) return e;
  }
  // Few of them and long: through rings (bf16: 32 of 1500 rows 11 us by rings, 21 by CTAs;
  // 128 of 1500 22 and 30, of 256 7.0 and 6.3; 320 of 1500 51 and 52).
  a.many = 0x7fffffff;
  if ((units < 160 && mean > 256) || (units < 320 && mean > 1024))
    return compact_ring<FMT>(a, units, s);
  // A lone long sequence among many short ones, in few layers, is too few CTAs: it goes
  // through rings behind the others (8200 rows of 8 heads in one layer among 60 sequences: 20
  // us, 111 without; in vain 2 to 3 us).
  const int64_t lone = (int64_t)a.kv.n * a.kv.Hkv;
  const bool rings = lone <= 64 && a.total > 4096;
  if (rings) a.many = a.total / 2;  // (one sequence at most keeps more)
  const int64_t grid = a.few > 0 ? min(units, (int64_t)152 * 4) : units;
  compact_cta_kernel<FMT><<<(unsigned)grid, NT, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !rings) return e;
  a.few = a.many;
  a.many = 0x7fffffff;
  return compact_ring<FMT>(a, lone, s);
}

}  // namespace

cudaError_t launch_kv_copy_pages(const CopyPagesArgs &a, cudaStream_t s) {
  const Parts x = parts_of(a.kv);
  const int64_t pages = (int64_t)a.n_pairs * a.kv.n;
  // By a warp, by a CTA, or in pieces (NVFP4, 446 pages of 146 vectors in 40 layers: 11 us by
  // warps, 53 in pieces; 391 of 876 vectors: 71 us by CTAs, 200 in pieces; E4M3, 96 of 8256
  // in 32 layers: 136 by CTAs, 120 in pieces; 4 pages of 2064 3.5 and 2.1).
  const bool many = pages > 152 * 4;
  if (many && x.all <= 512) {
    const int64_t grid = min((pages + NT / 32 - 1) / (NT / 32), (int64_t)152 * 4);
    copy_small_kernel<32><<<(unsigned)grid, NT, 0, s>>>(a);
  } else if (many && x.codes <= 2048) {
    copy_small_kernel<NT><<<(unsigned)min(pages, (int64_t)152 * 4), NT, 0, s>>>(a);
  } else {
    const int64_t each = (x.codes + kTogether * kPiece - 1) / (kTogether * kPiece);
    const int64_t grid = pages * (2 * each + (x.scales > 0));
    if (grid > 0x7fffffff) return cudaErrorNotYetImplemented;
    copy_pages_kernel<<<(unsigned)grid, NT, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(CompactArgs a, cudaStream_t s) {
  return a.kv.format == kKvBf16   ? compact_fmt<kKvBf16>(a, s)
         : a.kv.format == kKvE4m3 ? compact_fmt<kKvE4m3>(a, s)
                                  : compact_fmt<kKvNvfp4>(a, s);
}

}  // namespace attn_skip
