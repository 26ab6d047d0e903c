// What the two kernels over the paged cache share: waits, the tile of a CTA, the
// pages of a sequence.
#pragma once
#include <cuda.h>
#include <math.h>

#include "internal.h"
#include "tc_common.cuh"

namespace attn_skip {
namespace {

using namespace tc;

constexpr int D = 128;   // head size
constexpr int BN = 128;  // keys per block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;  // an exp reference may lag the max by 2^8
constexpr float kPLog2 = 7.0f;  // fp16 weights carry a factor 2^7: with the lag, up to fp16's 2^15

// The larger one, or a NaN if there is one (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The bounded waits of the other kernels with their slow path out of line (some
// forty waits share the instruction cache) and with sixteen tries between two
// looks at the abort flag and the clock (most warps wait most of the time, and
// the converters need the issue slots).
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort,
                                            unsigned *err) {
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait_shared(uint32_t bar, uint32_t parity, volatile int *abort,
                                                 unsigned *err) {
  return mbar_try_wait(bar, parity) || mbar_wait_slow(bar, parity, abort, err);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int c0, int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}

struct TileInfo {
  int s;          // sequence, -1: no tile for this CTA
  int t;          // tile of the sequence
  int tok0, ntok; // its first packed token, its tokens
  int pos0;       // position of its first token
  int kv;         // the end of the keys that some row of the tile sees
  int j0, nb;     // first block, blocks
  float ln_lam;   // -inf: dense, every block is kept
};

// ------------------------------------------------------------- tile of a CTA --
// Tiles run sequence by sequence, each sequence's last (longest) tile first.  Set-up
// code runs once a CTA from a cold instruction cache, so the common cases are
// kept short: where every chunk is at most one tile, CTA tile i is sequence i's;
// where there is one sequence, it is its; otherwise running sums over 32
// sequences at a time find it.
__device__ __forceinline__ int known_sequence(const ChunkArgs &a, int i) {
  return a.max_chunk <= a.TT ? i : a.n_seq == 1 ? 0 : -1;
}

// Length of a chunk, 0 where its bounds are bad (the sequence then has no tile).
__device__ __forceinline__ int chunk_of(const ChunkArgs &a, int c0, int c1, bool &bad) {
  if (c0 < 0 || c1 < c0 || c1 - c0 > a.max_chunk || c1 > a.total) {
    bad = true;
    return 0;
  }
  return c1 - c0;
}

// The tile with number i, for the whole warp; `known`: its sequence, or -1.  A bad
// cached length is an empty cache, a bad threshold 0.
__device__ __forceinline__ TileInfo locate(const ChunkArgs &a, int i, int split, int lane,
                                           int known) {
  bool bad = false;
  int s = known, first = 0;  // the sequence and the number of its first tile
  if (known < 0) {
#pragma unroll 1
    for (int b = 0; b < a.n_seq && s < 0; b += 32) {
      const int q = b + lane;
      int nt = 0;
      if (q < a.n_seq)
        nt = (chunk_of(a, __ldg(a.cu_seqlens + q), __ldg(a.cu_seqlens + q + 1), bad) + a.TT - 1) / a.TT;
      int upto = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      upto += first;
      const unsigned mine = __ballot_sync(0xffffffffu, i >= upto - nt && i < upto);
      if (mine) {
        const int l = __ffs(mine) - 1;
        s = b + l;
        first = __shfl_sync(0xffffffffu, upto - nt, l);
      } else {
        first = __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  TileInfo x{};
  x.s = -1;
  if (s < 0) return x;
  const int c0 = __ldg(a.cu_seqlens + s), c1 = __ldg(a.cu_seqlens + s + 1);
  int kv = __ldg(a.kv_len + s);
  const float lam = __ldg(a.lambda + s);
  const int len = chunk_of(a, c0, c1, bad);
  const int nt = (len + a.TT - 1) / a.TT;
  const int t = known < 0 || a.n_seq == 1 ? nt - 1 - (i - first) : 0;
  if (t < 0 || t >= nt) return x;
  if (kv < 0 || kv > a.max_kv) kv = 0;
  x.s = s;
  x.t = t;
  x.tok0 = c0 + t * a.TT;
  x.ntok = min(a.TT, len - t * a.TT);
  x.pos0 = kv - len + t * a.TT;
  // Rows behind the last key that some row of the tile sees (later tokens of the
  // chunk among them) may hold anything: they are not there for the tile.
  x.kv = a.causal ? max(0, x.pos0 + x.ntok) : kv;
  const int blocks = (x.kv + BN - 1) / BN;  // then this split's share of them
  x.j0 = split * a.bps;
  x.nb = max(0, min(blocks, x.j0 + a.bps) - x.j0);
  x.ln_lam = lam > 0.f && lam < 1.f ? logf(lam) : -INFINITY;
  return x;
}

// Reports the batch's bad bounds, lengths and thresholds; one warp of one CTA.
__device__ __noinline__ void check_batch(const ChunkArgs &a, int lane) {
  bool bad = false;
#pragma unroll 1
  for (int s = lane; s < a.n_seq; s += 32) {
    chunk_of(a, __ldg(a.cu_seqlens + s), __ldg(a.cu_seqlens + s + 1), bad);
    const int kv = __ldg(a.kv_len + s);
    const float lam = __ldg(a.lambda + s);
    bad |= kv < 0 || kv > a.max_kv || !(lam >= 0.f && lam < 1.f);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err, kErrBadArg);
}

// ------------------------------------------------------------------- pages --
// What a producer warp needs to copy blocks.  A part is a page, or 128 rows of a
// larger page; lane l holds the page id of part base + l, and the next 32 are
// loaded one window ahead.  A page id out of range is reported and page 0 read
// in its place.
struct Producer {
  const int32_t *table;  // the sequence's row; null: its rows are page `seq`
  int seq;
  int lsub, per_page;    // log2 of a part's rows, parts of a page
  int n_parts, base, cur, nxt, hk;
  uint64_t policy;
  bool bad;
};

__device__ __forceinline__ int page_of_part(const ChunkArgs &a, const Producer &p, int u) {
  if (!p.table) return p.seq;
  const int i = p.per_page == 1 ? u : (int)((unsigned)u / (unsigned)p.per_page);
  return i < a.max_pages ? __ldg(p.table + i) : 0;
}

// The first pages' ids load before the sequence's length is known (n_parts is set
// then): entries of its row of the table, whether or not they stand for pages.
__device__ __forceinline__ void producer_start(const ChunkArgs &a, Producer &p, int s, int j0,
                                               int hk, int lane) {
  p.table = a.page_table ? a.page_table + (int64_t)s * a.max_pages : nullptr;
  p.seq = s;
  p.lsub = a.pages.page_size < BN ? 31 - __clz(a.pages.page_size) : 7;
  p.per_page = a.pages.page_size < BN ? 1 : a.pages.page_size / BN;
  p.bad = false;
  p.hk = hk;
  // Keys and values are read again by the other tiles of the sequence, or once.
  p.policy = a.max_chunk > a.TT ? policy_evict_last() : policy_evict_first();
  p.base = (j0 << (7 - p.lsub)) & ~31;
  p.cur = page_of_part(a, p, p.base + lane);
  p.nxt = page_of_part(a, p, p.base + 32 + lane);
}

// A producer warp's set-up: its tile, and the pages' ids in flight as early as may be.
__device__ __forceinline__ TileInfo producer_tile(const ChunkArgs &a, Producer &p, int i, int split,
                                                  int hk, int lane) {
  const int known = known_sequence(a, i);
  if (known >= 0) producer_start(a, p, known, split * a.bps, hk, lane);
  const TileInfo x = locate(a, i, split, lane, known);
  if (known < 0 && x.s >= 0) producer_start(a, p, x.s, split * a.bps, hk, lane);
  p.n_parts = (x.kv + (1 << p.lsub) - 1) >> p.lsub;
  return x;
}

// A producer warp's set-up for the blocks of x from x.j0 on.
__device__ __forceinline__ void producer_at(const ChunkArgs &a, Producer &p, const TileInfo &x, int hk,
                                            int lane) {
  producer_start(a, p, x.s, x.j0, hk, lane);
  p.n_parts = (x.kv + (1 << p.lsub) - 1) >> p.lsub;
}

// The parts of block j for the lanes of the warp: lane l < n has part l's page and
// its first row in the page.  Whole warp.
struct Part {
  int n, page, slot;
};
__device__ __forceinline__ Part part_of(const ChunkArgs &a, Producer &p, int j, int lane) {
  const int u0 = j << (7 - p.lsub), b = u0 & ~31;
  if (b != p.base) {
    p.cur = b == p.base + 32 ? p.nxt : page_of_part(a, p, b + lane);
    p.base = b;
    p.nxt = page_of_part(a, p, b + 32 + lane);
  }
  Part x;
  x.n = min(1 << (7 - p.lsub), p.n_parts - u0);
  x.page = __shfl_sync(0xffffffffu, p.cur, (u0 - b + lane) & 31);
  if (lane < x.n && (x.page < 0 || x.page >= a.pages.n_pages)) {
    p.bad = true;
    x.page = 0;
  }
  x.slot = p.per_page == 1 ? 0 : (int)((unsigned)(u0 + lane) % (unsigned)p.per_page) << p.lsub;
  return x;
}

}  // namespace
}  // namespace attn_skip
