// Rows and pages of the paged cache moved as they are: whole pages copied, and the
// rows that a sequence keeps moved together, in the caches of all layers at once.
#include <stdint.h>
#include <stdlib.h>

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
struct RowAt {
  int from_page, from_slot, to_page, to_slot;  // from_page -1: nothing to move
};

template <int FMT> struct RowBytes {
  static constexpr int value = FMT == kKvBf16 ? 256 : FMT == kKvE4m3 ? 128 : 64;
};

// BOTH: the unit's rows are keys and values; else one of the two, by the unit's number,
// and 16 * LPR bytes of each row.
template <int FMT, int LPR, int GROUP, bool BOTH>
__global__ void __launch_bounds__(NT) compact_kernel(const __grid_constant__ CompactArgs a) {
  constexpr int VECS = RowBytes<FMT>::value / 16, PARTS = VECS / LPR;
  constexpr int KV = BOTH ? 2 : 1;
  constexpr int U = BOTH ? 2 : 4;                  // rows a thread loads at a time
  constexpr int CHUNK = GROUP / LPR * U;           // rows of the group
  constexpr int BATCH = GROUP == 32 ? 32 : 1024;
  constexpr int MINE = BATCH / GROUP;              // rows of the batch whose scales a thread moves
  constexpr int GROUPS = NT / GROUP;
  static_assert(BATCH % CHUNK == 0, "whole chunks");
  __shared__ RowAt rows_at[GROUPS][BATCH];
  const int g = threadIdx.x / GROUP, t = threadIdx.x % GROUP;
  RowAt *at = rows_at[g];
  auto sync = [&] {
    if constexpr (GROUP == 32) __syncwarp();
    else __syncthreads();
  };
  unsigned unit = blockIdx.x * GROUPS + g;
  auto next = [&](unsigned n) {
    const unsigned q = unit / n, r = unit - q * n;
    unit = q;
    return (int)r;
  };
  const int split = next((unsigned)a.splits), part = next(PARTS), w0 = next(3 - KV);
  const int h = next((unsigned)a.kv.Hkv), s = next((unsigned)a.n_seq), layer = (int)unit;
  if (layer >= a.kv.n) return;  // (whole groups)
  const int c0 = a.cu_keep[s], c1 = a.cu_keep[s + 1];
  if (c0 < 0 || c1 < c0 || c1 > a.total) {
    if (t == 0) atomicOr(a.err, kErrBadArg);
    return;
  }
  const int n = c1 - c0, start = a.start ? a.start[s] : 0;
  const int32_t *keep = a.keep + (a.per_head ? (int64_t)h * a.total : 0) + c0;
  const bool in_place = !a.out_table;
  const int32_t *from = a.table + (int64_t)s * a.max_pages;
  const int32_t *to = in_place ? from : a.out_table + (int64_t)s * a.out_max_pages;
  const int64_t from_room = (int64_t)a.max_pages * a.kv.page_size;
  const int64_t to_room = in_place ? from_room : (int64_t)a.out_max_pages * a.kv.page_size;
  const auto &l = a.kv.layer[layer];
  uint8_t *codes[KV], *scale[KV], *block[KV];
#pragma unroll
  for (int w = 0; w < KV; ++w) {
    const bool value = BOTH ? w == 1 : w0 == 1;
    codes[w] = (value ? l.v : l.k) + (part * LPR + t % LPR) * 16;
    scale[w] = value ? l.v_scale : l.k_scale;
    block[w] = value ? l.v_bs : l.k_bs;
  }
  const int head_row = h * a.kv.page_size, page_rows = a.kv.Hkv * a.kv.page_size;
  bool bad = false;
  for (int j0 = split * BATCH; j0 < n; j0 += a.splits * BATCH) {
    sync();  // the batch before is done with the places
    const int m = min(BATCH, n - j0);
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int b = t + i * GROUP;
      if (b >= m) break;
      const int64_t src = keep[j0 + b], dst = (int64_t)start + j0 + b;
      RowAt x{-1, 0, 0, 0};
      if (src < 0 || src >= from_room || dst < 0 || dst >= to_room || (in_place && src < dst)) {
        bad = true;
      } else if (!in_place || src != dst) {
        const unsigned ps = (unsigned)a.kv.page_size;
        const unsigned pf = a.kv.page_shift >= 0 ? (unsigned)src >> a.kv.page_shift : (unsigned)src / ps;
        const unsigned pt = a.kv.page_shift >= 0 ? (unsigned)dst >> a.kv.page_shift : (unsigned)dst / ps;
        x = RowAt{from[pf], (int)((unsigned)src - pf * ps), to[pt], (int)((unsigned)dst - pt * ps)};
        if (x.from_page < 0 || x.from_page >= a.kv.n_pages || x.to_page < 0 ||
            x.to_page >= a.kv.n_pages) {
          bad = true;
          x.from_page = -1;
        }
      }
      at[b] = x;
    }
    sync();
    uint8_t sc[MINE][KV];
    uint2 bs[MINE][KV];
    if (FMT != kKvBf16 && part == 0) {
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int b = t + i * GROUP;
        if (b >= m || at[b].from_page < 0) continue;
        const int64_t row = (int64_t)at[b].from_page * page_rows + head_row + at[b].from_slot;
#pragma unroll
        for (int w = 0; w < KV; ++w) {
          sc[i][w] = scale[w][row];
          if (FMT == kKvNvfp4) bs[i][w] = *reinterpret_cast<const uint2 *>(block[w] + row * 8);
        }
      }
    }
    auto load = [&](int c, uint4 (&x)[U][KV]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = c + t / LPR + u * (GROUP / LPR);
        if (b >= m || at[b].from_page < 0) continue;
        const int64_t byte = at[b].from_page * a.kv.page_stride +
                             (int64_t)(head_row + at[b].from_slot) * RowBytes<FMT>::value;
#pragma unroll
        for (int w = 0; w < KV; ++w) x[u][w] = *reinterpret_cast<const uint4 *>(codes[w] + byte);
      }
    };
    auto store = [&](int c, const uint4 (&x)[U][KV]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = c + t / LPR + u * (GROUP / LPR);
        if (b >= m || at[b].from_page < 0) continue;
        const int64_t byte = at[b].to_page * a.kv.page_stride +
                             (int64_t)(head_row + at[b].to_slot) * RowBytes<FMT>::value;
#pragma unroll
        for (int w = 0; w < KV; ++w) *reinterpret_cast<uint4 *>(codes[w] + byte) = x[u][w];
      }
    };
    uint4 x[U][KV], y[U][KV];
    load(0, x);
    for (int c = 0; c < m; c += 2 * CHUNK) {
      load(c + CHUNK, y);
      sync();  // all loads up to here come before the stores below
      if (FMT != kKvBf16 && part == 0 && c == 0) {
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          const int b = t + i * GROUP;
          if (b >= m || at[b].from_page < 0) continue;
          const int64_t row = (int64_t)at[b].to_page * page_rows + head_row + at[b].to_slot;
#pragma unroll
          for (int w = 0; w < KV; ++w) {
            scale[w][row] = sc[i][w];
            if (FMT == kKvNvfp4) *reinterpret_cast<uint2 *>(block[w] + row * 8) = bs[i][w];
          }
        }
      }
      store(c, x);
      load(c + 2 * CHUNK, x);
      sync();
      store(c + CHUNK, y);
    }
  }
  if (bad) atomicOr(a.err, kErrBadArg);
}

template <int FMT, int LPR, int GROUP, bool BOTH>
cudaError_t compact_launch(const CompactArgs &a, cudaStream_t s) {
  constexpr int PER_HEAD = RowBytes<FMT>::value / 16 / LPR * (BOTH ? 1 : 2);
  constexpr int GROUPS = NT / GROUP;
  const int64_t units = (int64_t)a.kv.n * a.n_seq * a.kv.Hkv * PER_HEAD * a.splits;
  if (units > 0x7fffffff) return cudaErrorNotYetImplemented;
  compact_kernel<FMT, LPR, GROUP, BOTH><<<(unsigned)((units + GROUPS - 1) / GROUPS), NT, 0, s>>>(a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t compact_fmt(CompactArgs &a, cudaStream_t s) {
  constexpr int VECS = RowBytes<FMT>::value / 16;
  const int64_t units = (int64_t)a.kv.n * a.n_seq * a.kv.Hkv;
  const int64_t mean = a.total / a.n_seq;
  a.splits = 1;
  if (mean <= 64) return compact_launch<FMT, VECS, 32, true>(a, s);
  if (!a.out_table) {
    // In place a (layer, sequence, head) goes through its rows in order; where these are
    // few, keys and values are cut into columns of 32 (64) bytes.
    if (units * 2 < 152 * 8 && !getenv("NOCUT")) return compact_launch<FMT, VECS == 4 ? 2 : VECS / 4, NT, false>(a, s);
    return compact_launch<FMT, VECS, NT, false>(a, s);
  }
  // Rows may be shared out where none is overwritten.
  while (a.splits < 64 && units * 2 * a.splits < 152 * 8 && mean / a.splits > 1024) a.splits *= 2;
  return compact_launch<FMT, VECS, NT, false>(a, s);
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
