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
  int kv;         // the sequence's cached length
  int j0, nb;     // first block, blocks
  float ln_lam;   // -inf: dense, every block is kept
};

// ------------------------------------------------------------- tile of a CTA --
// Tiles run sequence by sequence, each sequence's last (longest) tile first;
// one warp locates tile i by running sums over 32 sequences at a time.
__device__ __noinline__ void locate(const ChunkArgs &a, int i, int split, int lane, bool report,
                                    TileInfo *out) {
  bool bad = false, found = false;
  int before = 0;
#pragma unroll 1
  for (int b = 0; b < a.n_seq && (report || !found); b += 32) {
    const int s = b + lane;
    int c0 = 0, len = 0, kv = 0;
    float lam = 0.f;
    if (s < a.n_seq) {
      c0 = __ldg(a.cu_seqlens + s);
      const int c1 = __ldg(a.cu_seqlens + s + 1);
      kv = __ldg(a.kv_len + s);
      lam = __ldg(a.lambda + s);
      len = c1 - c0;
      // Bad bounds: the sequence has no tile.  A bad cached length: an empty
      // cache.  A bad threshold: 0.
      if (c0 < 0 || c1 < c0 || len > a.max_chunk || c1 > a.total) { len = 0; bad = true; }
      if (kv < 0 || kv > a.max_kv) { kv = 0; bad = true; }
      if (!(lam >= 0.f && lam < 1.f)) { lam = 0.f; bad = true; }
    }
    const int nt = (len + a.TT - 1) / a.TT;
    int upto = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    upto += before;
    if (!found && i >= upto - nt && i < upto) {
      TileInfo x;
      x.s = s;
      x.t = upto - 1 - i;
      x.tok0 = c0 + x.t * a.TT;
      x.ntok = min(a.TT, len - x.t * a.TT);
      x.pos0 = kv - len + x.t * a.TT;
      x.kv = kv;
      // Keys that some row of the tile sees, then this split's blocks of them.
      const int seen = a.causal ? max(0, x.pos0 + x.ntok) : kv;
      const int blocks = (seen + BN - 1) / BN;
      x.j0 = split * a.bps;
      x.nb = max(0, min(blocks, x.j0 + a.bps) - x.j0);
      x.ln_lam = lam > 0.f ? logf(lam) : -INFINITY;
      *out = x;
      found = true;
    }
    found = __any_sync(0xffffffffu, found);
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  if (!found && lane == 0) out->s = -1;
  if (report && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err, kErrBadArg);
  __syncwarp();
}

// ------------------------------------------------------------------- pages --
// What a producer warp needs to copy blocks.  A part is a page, or 128 rows of a
// larger page; lane l holds the page id of part base + l, and the next 32 are
// loaded one window ahead.  A page id out of range is reported and page 0 read
// in its place.
struct Producer {
  const int32_t *table;  // the sequence's row; null: its rows are page `seq`
  int seq;
  int sub, per_page;     // rows of a part, parts of a page
  int n_parts, base, cur, nxt, hk;
  uint64_t policy;
  bool bad;
};

__device__ __forceinline__ int page_of_part(const ChunkArgs &a, Producer &p, int u) {
  if (u >= p.n_parts) return 0;
  if (!p.table) return p.seq;
  const int id = __ldg(p.table + (unsigned)u / (unsigned)p.per_page);
  if (id < 0 || id >= a.pages.n_pages) {
    p.bad = true;
    return 0;
  }
  return id;
}

__device__ __forceinline__ void producer_init(const ChunkArgs &a, Producer &p, const TileInfo &x, int hk,
                                           int lane) {
  p.table = a.page_table ? a.page_table + (int64_t)x.s * a.max_pages : nullptr;
  p.seq = x.s;
  p.sub = min(a.pages.page_size, BN);
  p.per_page = a.pages.page_size / p.sub;
  p.n_parts = (x.kv + p.sub - 1) / p.sub;
  p.bad = false;
  p.hk = hk;
  // Keys and values are read again by the other tiles of the sequence, or once.
  p.policy = a.max_chunk > a.TT ? policy_evict_last() : policy_evict_first();
  p.base = (x.j0 * (BN / p.sub)) & ~31;
  p.cur = page_of_part(a, p, p.base + lane);
  p.nxt = page_of_part(a, p, p.base + 32 + lane);
}

// The parts of block j for the lanes of the warp: lane l < n has part l's page and
// its first row in the page.  Whole warp.
struct Part {
  int n, page, slot;
};
__device__ __forceinline__ Part part_of(const ChunkArgs &a, Producer &p, int j, int lane) {
  const int ppb = BN / p.sub, u0 = j * ppb, b = u0 & ~31;
  if (b != p.base) {
    p.cur = b == p.base + 32 ? p.nxt : page_of_part(a, p, b + lane);
    p.base = b;
    p.nxt = page_of_part(a, p, b + 32 + lane);
  }
  Part x;
  x.n = min(ppb, p.n_parts - u0);
  x.page = __shfl_sync(0xffffffffu, p.cur, (u0 - b + lane) & 31);
  x.slot = (int)((unsigned)(u0 + lane) % (unsigned)p.per_page) * p.sub;
  return x;
}

}  // namespace
}  // namespace attn_skip
