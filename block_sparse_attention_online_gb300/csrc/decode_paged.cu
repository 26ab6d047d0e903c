// Decode over the quantised paged caches: attention of tiles of at most eight
// rows (query heads of a KV head times new tokens) over E4M3 or NVFP4 pages, with
// softmax-threshold block skipping (d = 128, 128-key blocks), on warp-level
// m16n8k16 products.
//
// The mathematics is that of the chunk kernel (a tile of few rows of it).  Here
// the keys are the 16 rows of a product and the tile's rows its 8 columns, so
// codes go from shared memory to fp16 operand registers (one cvt per two codes)
// and a row scale multiplies one score instead of 128 elements:
//   S^T = K Q^T        A = codes of 16 keys, B = fp16 queries (2^x scaled)
//   s_c = S_c * scale * 2^(e_k,c - x)         (log2 units)
//   w_c = 2^(s_c - sref),  sref the running max of s_c of the warp
//   P_c = w_c 2^e_v,c 2^x,  x = sref - ref + 7, ref the running max of s_c + e_v,c
//   O^T += V^T P       A = codes of 16 keys, transposed by byte pairs, B = P
//   l += w_c
// An NVFP4 code times its block scale is an fp16 (exact); P is rounded to fp16.
// The references may lag by 2^8, so with 2^7 P stays below fp16's 2^16, has its 11
// bits down to 2^-21 of the largest contribution and steps of 2^-31 of it below
// (it counts where the row with the large weight holds a zero).  A row of zeros has
// no part in ref (2^e_v,c counts as 0).  Two references, since the values' exponents
// span as much as fp32's: with ref alone the weights of rows of small values, or of
// zeros, were lost beside rows of large ones.
//
// One CTA per (sequence, KV head, split), two on an SM; where these are more than
// fit, the CTAs share the blocks out (below).  Eight warps share each 128-key block,
// 16 keys a warp, each with its own running reference, row sums and outputs, merged
// at the end as splits are; two more warps fetch keys and values through TMA rings
// (two CTAs hold about 200 KB of cache in flight), on into a CTA's next tile while
// the last one is merged.
// Why not tcgen05: its operands come from shared memory, and writing a block's
// 64 KB there as fp16 costs more issue slots than the cache costs bandwidth
// (16 sequences of 32768 tokens, E4M3: 418 us on that path).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace attn_skip {
namespace {

using namespace tc;

constexpr int NCW = 8;            // compute warps
constexpr int WARP_K = NCW, WARP_V = NCW + 1;
constexpr int NT = (NCW + 2) * 32;
constexpr int ROWS = 8;           // rows of a tile (columns of the products)
constexpr int NDEC = 4;           // decision ring
constexpr int kVoteBarrier = 1;
constexpr int MERGE_COLS = 32;
constexpr unsigned kCtas = 2 * 152;  // two on each SM
constexpr float kNoRef = -3e38f;     // sref of a row without a key so far
constexpr float kBelow = 118.f;      // ref stays above sref - 118: x and what undoes it are normal

template <int FMT> struct Cfg;
template <> struct Cfg<kKvE4m3> {
  static constexpr int NST = 3;  // stages of keys, and of values
  static constexpr uint32_t ROW = D, BS = 0;
};
template <> struct Cfg<kKvNvfp4> {
  static constexpr int NST = 5;
  static constexpr uint32_t ROW = D / 2, BS = BN * D / 16;
};
template <int FMT> struct Layout {
  using C = Cfg<FMT>;
  static constexpr uint32_t CODES = BN * C::ROW;
  // Code tiles first (1024-byte aligned), then block scales and row scales: a
  // key stage also has the row scales of its values, needed before they are.
  static constexpr uint32_t K = 0, V = K + C::NST * CODES, KX = V + C::NST * CODES;
  static constexpr uint32_t KXS = C::BS + 2 * BN, VX = KX + C::NST * KXS;
  static constexpr uint32_t MERGE = VX + C::NST * C::BS;
  static constexpr uint32_t END = MERGE + NCW * ROWS * (MERGE_COLS + 4) * 4;
};

// A run of blocks of one tile (x.s = -1: none) and where its result goes.
struct Item {
  TileInfo x;
  int hk, slot;  // KV head; slot of the partial
  int fill;      // one more than the last slot to mark as empty besides, or 0
};

struct Shared {
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
  uint64_t dec_full[NDEC], dec_empty[NDEC];
  uint64_t item_full[2], item_empty[2];
  int dec[NDEC];
  float rmax[2][NCW][ROWS];        // row maxima of the warps' keys, blocks of either parity
  float ml[3][NCW][ROWS];          // the warps' ref - 7, row sums and sref
  Item item[2];                    // ring of the CTA's work
  uint32_t word;                   // the bitmap's current word
  int abort;
};
static_assert(2 * (Layout<kKvE4m3>::END + sizeof(Shared) + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(2 * (Layout<kKvNvfp4>::END + sizeof(Shared) + 1024) <= 228 * 1024, "two CTAs an SM");

// Key of the warp's sixteen that is row m of its products: chosen so that the
// eight lanes of a 16-byte load (and the sixteen of an 8-byte load) meet
// different banks of the swizzled tiles, for the key reads (rows m) and the
// transposed value reads (rows 2 t, 2 t + 1, ..).
template <int FMT> __device__ __forceinline__ int key_of(int m) {
  if constexpr (FMT == kKvE4m3) return m;
  const int b0 = m & 1, b1 = (m >> 1) & 1;
  return (m & 12) | (b0 << 1) | (b1 ^ b0);
}

// Byte address of 16-byte chunk c of row r of a swizzled code tile.
template <int FMT> __device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
  if constexpr (FMT == kKvE4m3) return tile + r * 128 + ((c ^ (r & 7)) << 4);
  return tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival on `bar` once its cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Block j's rows into stage buffers; whole warp.  Codes by TMA (swizzled), part
// by part, one lane a part; scales in 16-byte pieces by cp.async of all lanes (a
// bulk copy a part for each of them made pages of 16 rows half again as slow:
// 48 copies a block).  `full` takes the byte count's arrival and, where there
// are scales, one of each lane.
template <int FMT>
__device__ __forceinline__ void load_block(const ChunkArgs &a, Producer &p, const CUtensorMap *map,
                                           bool value, int j, uint32_t codes, uint32_t extra,
                                           uint32_t full, int lane) {
  using C = Cfg<FMT>;
  const int sub = 1 << p.lsub;
  const Part x = part_of(a, p, j, lane);
  const int rows = x.n * sub;  // rows of the block in the cache's pages
  const KvPages &g = a.pages;
  if (lane == 0) mbar_expect_tx(full, rows * C::ROW);
  __syncwarp();
  if (lane < x.n)
    tma_load_4d(codes + lane * sub * C::ROW, map, full, 0, x.slot, p.hk, x.page, p.policy);
  // Scale index of row r of the block: that of its part's first row, and on.
  const int64_t first = ((int64_t)x.page * g.Hkv + p.hk) * g.page_size + x.slot;
  auto row_at = [&](int r) { return __shfl_sync(0xffffffffu, first, r >> p.lsub) + (r & (sub - 1)); };
  if constexpr (FMT == kKvNvfp4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * (lane + 32 * i);
      const int64_t at = row_at(r);
      if (r < rows) cp_async16(extra + r * 8, (value ? g.v_bs : g.k_bs) + at * 8);
    }
  }
  if (!value) {
    const int r = 16 * (lane & 7);
    const int64_t at = row_at(r);
    if (lane < 16 && r < rows)
      cp_async16(extra + C::BS + (lane < 8 ? 0 : BN) + r, (lane < 8 ? g.k_scale : g.v_scale) + at);
  }
  if (!value || FMT == kKvNvfp4) cp_async_arrive(full);
  __syncwarp();
}

// Whether value row r of a block with `left` rows to kv, of scale byte `byte`, holds
// zeros, to which the writer gives byte 127.  The row's four lanes look at a quarter
// of its codes each.
template <int FMT>
__device__ __noinline__ bool zero_row(const ChunkArgs &a, const Item &item, int r, int left,
                                      uint32_t byte, int t) {
  const KvPages &p = a.pages;
  constexpr uint32_t QUARTER = Cfg<FMT>::ROW / 4;
  const bool mine = byte == 127u && r < left;
  const int pos = item.x.kv - left + r;
  uint32_t any = 0;
  if (mine) {
    int page = __ldg(a.page_table + (int64_t)item.x.s * a.max_pages + pos / p.page_size);
    if (page < 0 || page >= p.n_pages) page = 0;
    const uint4 *c = reinterpret_cast<const uint4 *>(
        (const uint8_t *)p.v + page * p.page_stride +
        ((int64_t)item.hk * p.page_size + pos % p.page_size) * Cfg<FMT>::ROW + t * QUARTER);
#pragma unroll
    for (uint32_t k = 0; k < QUARTER / 16; ++k) {
      const uint4 w = __ldg(c + k);
      any |= w.x | w.y | w.z | w.w;
    }
    any &= FMT == kKvE4m3 ? 0x7f7f7f7fu : 0x77777777u;
  }
  any |= __shfl_xor_sync(0xffffffffu, any, 1);
  any |= __shfl_xor_sync(0xffffffffu, any, 2);
  return mine && any == 0;
}

// ------------------------------------------------------- shares of a batch --
// With more pieces (sequence, KV head, split) than the chip has room for, the grid
// is what it has room for and the CTAs share the work out among themselves, from
// the lengths that only the device knows.  Where every tile is dense its blocks are
// one list, sequence by sequence and head by head, cut into equal runs (a tile may
// be cut anywhere; its partials take the slots in order); otherwise the list is of
// the pieces that have blocks, whose bounds the running maxima need, and a CTA
// takes every gridDim.x-th.  24 sequences of 8192 to 32768 tokens, NVFP4: 153 us,
// 189 with a CTA a piece; E4M3 152 and 170.  (16 sequences of one length, E4M3, bound
// by memory: 178 and 172, since equal runs do not follow the SMs' different distances
// to memory; two or three rounds of shorter runs cost more than they bring.  Whole
// pieces the hardware's scheduler spreads better, but the host cannot tell which
// batches have thresholds: NVFP4 261 us against the list's 280, E4M3 238 and 252;
// whole tiles, one split, are left to it: 100 sequences of up to 4000, NVFP4, 104 us
// and 121.)
constexpr int SEQS = 4;  // sequences a lane keeps: up to 128

struct Plan {  // (32 sequences at a time: mostly there are no more)
  unsigned nb[SEQS];    // blocks of sequences lane, lane + 32, ..
  unsigned at[SEQS];    // the first list entry of each
  unsigned pos, end;    // this CTA's next entry, the entries' (or its run's) end
  unsigned unit;        // entries of a run; 0: the list is of pieces
};

// Entries of a tile of nb blocks.
__device__ __forceinline__ unsigned entries_of(const ChunkArgs &a, bool runs, unsigned nb) {
  return runs ? nb : (nb + a.bps - 1) / a.bps;
}

// One warp; also marks the partials of the sequences without a visible key.
__device__ __noinline__ void plan_start(const ChunkArgs &a, Plan &p, int lane) {
  bool cut = true, none[SEQS], bad = false;
  unsigned longest = 0;
  const int chunks = (a.n_seq + 31) / 32;
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    const int s = 32 * i + lane;
    p.nb[i] = 0;
    none[i] = false;
    if (s >= a.n_seq) continue;
    const int len = chunk_of(a, __ldg(a.cu_seqlens + s), __ldg(a.cu_seqlens + s + 1), bad);
    const int kv = __ldg(a.kv_len + s);
    const float lam = __ldg(a.lambda + s);
    if (len == 0) continue;
    p.nb[i] = kv < 0 || kv > a.max_kv ? 0u : (unsigned)(kv + BN - 1) / BN;
    none[i] = p.nb[i] == 0;
    cut = cut && !(lam > 0.f && lam < 1.f);
    longest = max(longest, p.nb[i]);
  }
  cut = __all_sync(0xffffffffu, cut);
  longest = __reduce_max_sync(0xffffffffu, longest);
  unsigned all = 0;
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    const unsigned w = entries_of(a, cut, p.nb[i]) * (unsigned)a.Hkv;
    unsigned upto = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    p.at[i] = all + upto - w;
    all += __shfl_sync(0xffffffffu, upto, 31);
  }
  p.unit = 0;
  p.pos = blockIdx.x;
  p.end = all;
  if (cut) {
    // A tile of n blocks meets at most ceil((n - 1) / unit) + 1 runs: no more than
    // it has slots.
    const unsigned slots = a.n_splits - 1;
    p.unit = max(max((all + gridDim.x - 1) / gridDim.x, (longest + slots - 1) / slots), 1u);
    // (Runs past the list's end start behind it; the product stays below 2^32.)
    p.pos = min(all, blockIdx.x * p.unit);
    p.end = min(all, p.pos + p.unit);
  }
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    unsigned m = __ballot_sync(0xffffffffu, none[i]);
#pragma unroll 1
    for (; m; m &= m - 1) {
      const int s = 32 * i + __ffs(m) - 1;
      if (s % gridDim.x != blockIdx.x) continue;
      const int64_t r0 = (int64_t)__ldg(a.cu_seqlens + s) * a.Hq;
      const int64_t n = (int64_t)__ldg(a.cu_seqlens + s + 1) * a.Hq - r0;
      for (int64_t r = lane; r < n * a.n_splits; r += 32) a.lse_part[r0 * a.n_splits + r] = -INFINITY;
    }
  }
}

// The CTA's next item; whole warp.
__device__ __noinline__ Item plan_next(const ChunkArgs &a, Plan &p, int lane) {
  Item y{};
  y.x.s = -1;
  if (p.pos >= p.end) return y;
  const bool runs = p.unit != 0;
  unsigned nb = 0, at = 0;
  int s = -1;
#pragma unroll 1
  for (int i = 0; 32 * i < a.n_seq && s < 0; ++i) {
    const unsigned w = entries_of(a, runs, p.nb[i]) * (unsigned)a.Hkv;
    const unsigned m = __ballot_sync(0xffffffffu, p.pos - p.at[i] < w);  // (below: wraps)
    if (!m) continue;
    const int l = __ffs(m) - 1;
    s = 32 * i + l;
    nb = __shfl_sync(0xffffffffu, p.nb[i], l);
    at = __shfl_sync(0xffffffffu, p.at[i], l);
  }
  if (s < 0) return y;  // (the list has every entry below its end)
  const unsigned per = entries_of(a, runs, nb), h = (p.pos - at) / per, r = p.pos - at - h * per;
  y.hk = (int)h;
  unsigned j0 = r, n, slots;  // blocks from j0 on; slots of the tile that have a partial
  if (runs) {
    const unsigned first = (p.pos - r) / p.unit;  // the run in which the tile starts
    n = min(nb - r, p.end - p.pos);
    y.slot = (int)(p.pos / p.unit - first);
    slots = (unsigned)y.slot + 1;
    p.pos += n;
  } else {
    j0 = r * (unsigned)a.bps;
    n = min((unsigned)a.bps, nb - j0);
    y.slot = (int)r;
    slots = per;
    p.pos += gridDim.x;
  }
  y.fill = j0 + n == nb && slots < (unsigned)a.n_splits ? a.n_splits : 0;
  const int c0 = __ldg(a.cu_seqlens + s);
  const float lam = __ldg(a.lambda + s);
  y.x.s = s;
  y.x.t = 0;
  y.x.tok0 = c0;
  y.x.ntok = __ldg(a.cu_seqlens + s + 1) - c0;
  y.x.kv = __ldg(a.kv_len + s);
  y.x.pos0 = y.x.kv - y.x.ntok;
  y.x.j0 = (int)j0;
  y.x.nb = (int)n;
  y.x.ln_lam = lam > 0.f && lam < 1.f ? logf(lam) : -INFINITY;
  return y;
}

template <int FMT>
__global__ void __launch_bounds__(NT, 2)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ ChunkArgs a) {
  using C = Cfg<FMT>;
  using L = Layout<FMT>;
  constexpr int NST = C::NST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw + L::END);
  const uint32_t base = smem_u32(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (base & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (tid == 0) atomicOr(a.err, kErrLayout);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits for this grid's end)
  volatile int *abort = &sh.abort;
  auto wait_warp = [&](uint64_t *b, int phase) {
    return __all_sync(0xffffffffu, mbar_wait_shared(smem_u32(b), phase & 1, abort, a.err));
  };

  if (tid == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), 1 + 32);
      mbar_init(smem_u32(&sh.v_full[i]), FMT == kKvNvfp4 ? 1 + 32 : 1);
      mbar_init(smem_u32(&sh.k_empty[i]), NCW);
      mbar_init(smem_u32(&sh.v_empty[i]), NCW);
    }
    for (int i = 0; i < NDEC; ++i) {
      mbar_init(smem_u32(&sh.dec_full[i]), 1);
      mbar_init(smem_u32(&sh.dec_empty[i]), 1);  // the value producer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.item_full[i]), 1);
      mbar_init(smem_u32(&sh.item_empty[i]), NCW + 1);  // the value producer too
    }
    sh.abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  Producer pages;  // of the two producer warps
  Plan plan;       // of the key producer
  if (warp >= WARP_K) {
    if (a.shared_out) {
      if (warp == WARP_K) {
        plan_start(a, plan, lane);
        const Item y = plan_next(a, plan, lane);
        if (lane == 0) sh.item[0] = y;
      }
    } else {
      const int sp = (int)(blockIdx.x % a.n_splits);
      const int hk = (int)(blockIdx.x / a.n_splits) % a.Hkv;
      const TileInfo t = producer_tile(a, pages, (int)(blockIdx.x / a.n_splits / a.Hkv), sp, hk, lane);
      if (warp == WARP_K && lane == 0) sh.item[0] = Item{t, hk, sp, 0};
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && warp == WARP_V) check_batch(a, lane);
  if (!a.shared_out) {
    const Item &y = sh.item[0];
    if (y.x.s < 0) return;
    if (y.x.nb == 0) {  // no visible key: O = 0, LSE = -inf (one split), or a partial of no weight
      const int rows = y.x.ntok * a.G;
      for (int i = tid; i < rows * (D / 8); i += NT) {
        const int r = i / (D / 8);
        const int64_t orow = (int64_t)(y.x.tok0 + r / a.G) * a.Hq + y.hk * a.G + r % a.G;
        if (a.n_splits == 1)
          reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + orow * D)[i % (D / 8)] =
              make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0)
          (a.n_splits == 1 ? a.lse : a.lse_part)[orow * a.n_splits + y.slot] = -INFINITY;
      }
      return;
    }
  }

  if (warp >= WARP_K) {
    // ----------------------------------------------------------- producers --
    const bool value = warp == WARP_V;
    fence_proxy_async_smem();  // the barriers, for every lane's copies
    uint64_t *full = value ? sh.v_full : sh.k_full, *empty = value ? sh.v_empty : sh.k_empty;
    int n = 0, dc = 0;  // blocks fetched, decisions taken
#pragma unroll 1
    for (int it = 0; !*abort; ++it) {
      // The key producer finds the items (the first is there), the others follow.
      if (value) {
        if (it > 0 && !wait_warp(&sh.item_full[it & 1], it >> 1)) break;
      } else if (it > 0) {
        Item y{};
        y.x.s = -1;
        if (a.shared_out) y = plan_next(a, plan, lane);
        if (it >= 2 && !wait_warp(&sh.item_empty[it & 1], (it >> 1) - 1)) break;
        if (lane == 0) sh.item[it & 1] = y;
        __syncwarp();
      }
      if (!value && lane == 0) mbar_arrive(smem_u32(&sh.item_full[it & 1]));
      const TileInfo x = sh.item[it & 1].x;
      const int hk = sh.item[it & 1].hk;
      __syncwarp();
      if (value && lane == 0) mbar_arrive(smem_u32(&sh.item_empty[it & 1]));
      if (x.s < 0) break;
      const bool dense = x.ln_lam == -INFINITY;
      if (a.shared_out) producer_at(a, pages, x, hk, lane);
#pragma unroll 1
      for (int c = 0; c < x.nb && !*abort; ++c) {
        if (value && !dense) {  // (a dense tile keeps every block)
          const int d = dc++;
          if (!wait_warp(&sh.dec_full[d % NDEC], d / NDEC)) break;
          const int keep = sh.dec[d % NDEC];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.dec_empty[d % NDEC]));
          if (!keep) continue;
        }
        const int s = n % NST;
        if (n >= NST && !wait_warp(&empty[s], n / NST - 1)) break;
        load_block<FMT>(a, pages, value ? &tm_v : &tm_k, value, x.j0 + c,
                        base + (value ? L::V : L::K) + s * L::CODES,
                        base + (value ? L::VX + s * C::BS : L::KX + s * L::KXS), smem_u32(&full[s]),
                        lane);
        ++n;
      }
      if (!value && __any_sync(0xffffffffu, pages.bad) && lane == 0) atomicOr(a.err, kErrBadArg);
    }
    if (lane == 0) {  // the last load of each stage has landed before exit
#pragma unroll 1
      for (int s = 0; s < NST && s < n; ++s)
        mbar_wait_drain(smem_u32(&full[s]), ((s + ((n - 1 - s) / NST) * NST) / NST) & 1);
    }
    return;
  }

  // ------------------------------------------------------------ computation --
  // Lane (g, t): products' row g (and g + 8), columns 2 t, 2 t + 1.
  const int g = lane >> 2, t = lane & 3;
  const int k0 = warp * 16;  // the warp's keys of a block
  const int kr0 = k0 + key_of<FMT>(g), kr1 = kr0 + 8;
  // Values: keys of k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9; dims 16 g .. 16 g + 15, of
  // which 16 g + 2 i is row g of m-tile i and 16 g + 2 i + 1 its row g + 8.
  const int vr0 = k0 + key_of<FMT>(2 * t), vr1 = k0 + key_of<FMT>(2 * t + 1);
  bool ok = true;
  int kn = -1, vn = 0;  // stages (modulo 2 NST: with their phases)
  int decided = 0;      // blocks decided on before the item
#pragma unroll 1
  for (int it = 0;; ++it) {
    if (it > 0) {
      ok = wait_warp(&sh.item_full[it & 1], it >> 1);
      if (bar_red_or(kVoteBarrier, NCW * 32, !ok)) return;  // (all of them, or none)
    }
    const Item &item = sh.item[it & 1];
    const TileInfo x = item.x;
    if (x.s < 0) break;
    const int rows = x.ntok * a.G;
    const bool dense = x.ln_lam == -INFINITY;
    // Queries: row n = g of the tile, dims 32 t .. 32 t + 31; in k-step s, k = 2 t,
    // 2 t + 1 are dims 32 t + 4 s, + 1 and k = 2 t + 8, + 9 are + 2, + 3.
    uint32_t qf[16];
    float qs[2];  // scale * log2(e) * 2^-x of rows 2 t, 2 t + 1
    int rel[2];   // these rows see keys below kv + rel
    {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
      if (g < rows) {
        const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q + (int64_t)(x.tok0 + g / a.G) * a.q_tok_stride +
                                 (item.hk * a.G + g % a.G) * D + 32 * t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q) + i);
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      }
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        m = fmaxf(m, fmaxf(isfinite(lo) ? fabsf(lo) : 0.f, isfinite(hi) ? fabsf(hi) : 0.f));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // The largest 2^e with max|q| 2^e <= 2^15.
      const int b = __float_as_int(m);
      int e = 15 + 127 - (b >> 23) - ((b & 0x7fffff) != 0 ? 1 : 0);
      e = m > 0.f ? min(e, 100) : 0;
      const float f = __int_as_float((e + 127) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        qf[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
      const float mine = a.scale * kLog2e * __int_as_float((127 - e) << 23);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[i] = __shfl_sync(0xffffffffu, mine, (2 * t + i) * 4);
        rel[i] = a.causal && 2 * t + i < rows ? (2 * t + i) / a.G + 1 - x.ntok : 0;
      }
    }
    const int min_rel = a.causal ? 1 - x.ntok : 0;

    float o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // sref (whole numbers: sums with them are exact), 2^x, row sum.
    float sref[2] = {kNoRef, kNoRef}, px[2] = {1.f, 1.f}, l[2] = {0.f, 0.f};
    auto x_of = [](float f) { return (float)((__float_as_int(f) >> 23) - 127); };  // of f = 2^x
    float m2[2] = {-INFINITY, -INFINITY};  // running max of the split (log2 units), with a threshold
    int left = x.kv - x.j0 * BN + BN;      // rows below kv from the block on
    // With a threshold, a block's product with its values comes after the next block's
    // scores: between the decision to keep a block and the use of its values lies a
    // block's time, in which they arrive (16 sequences of 32768 tokens, E4M3, lambda
    // 1e-3: 221 us, 301 without, before the row sums' own reference; 220 with it).
    // Dense, the same takes 178: the vote, an exchange of all warps a block, costs more
    // than the values that it saves.  A dense tile has its values in time anyway.
    uint32_t b0 = 0, b1 = 0;  // P of the product to come
    bool pending = false;
    auto blocks = [&](auto threshold) {
      constexpr bool LATE = decltype(threshold)::value;
#pragma unroll 1
      for (int c = 0; c < item.x.nb + (LATE ? 1 : 0); ++c) {
        left -= BN;
        bool fresh = false;
        uint32_t n0 = 0, n1 = 0;
        if (!LATE || c < item.x.nb) {
          kn = kn == 2 * NST - 1 ? 0 : kn + 1;
          const int s = kn < NST ? kn : kn - NST;
          // After a failed wait the loop runs on (every later wait fails at once), so
          // that the warps meet the vote barriers equally often.
          if (ok) ok = wait_warp(&sh.k_full[s], kn >= NST);
          float p[2][2];        // [key g, g + 8][row 2 t, 2 t + 1]: scores, then P
          float vf[2];          // 2^e_v, the keys' value scales; 0 for rows of zeros
          bool nan_rows = false;
          {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t kx = base + L::KX + s * L::KXS, kt = base + L::K + s * L::CODES;
            if constexpr (FMT == kKvE4m3) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 u = lds128(chunk_at<FMT>(kt, kr0, 2 * t + h));
                const uint4 v = lds128(chunk_at<FMT>(kt, kr1, 2 * t + h));
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t a0, a1, a2, a3;
                  e4m3x4(uw[i], a0, a2);
                  e4m3x4(vw[i], a1, a3);
                  const int st = 4 * h + i;
                  mma16816(acc, a0, a1, a2, a3, qf[2 * st], qf[2 * st + 1]);
                }
              }
            } else {
              const uint4 u = lds128(chunk_at<FMT>(kt, kr0, t)), v = lds128(chunk_at<FMT>(kt, kr1, t));
              const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
              uint32_t us[2], vs[2];  // the scales of the lane's two blocks of sixteen, as pairs
              {
                const uint32_t b0 = lds16(kx + kr0 * 8 + 2 * t), b1 = lds16(kx + kr1 * 8 + 2 * t);
                e4m3x4(__byte_perm(b0, 0, 0x1100), us[0], us[1]);
                e4m3x4(__byte_perm(b1, 0, 0x1100), vs[0], vs[1]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // eight elements of a row: two k-steps
                uint32_t x0[4], x1[4];
                e2m1x8(uw[i], x0);
                e2m1x8(vw[i], x1);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  x0[k] = mul_f16x2(x0[k], us[i >> 1]);
                  x1[k] = mul_f16x2(x1[k], vs[i >> 1]);
                }
                mma16816(acc, x0[0], x1[0], x0[1], x1[1], qf[4 * i], qf[4 * i + 1]);
                mma16816(acc, x0[2], x1[2], x0[3], x1[3], qf[4 * i + 2], qf[4 * i + 3]);
              }
            }
            const uint32_t sc = kx + C::BS;
            const uint32_t eb0 = lds8(sc + kr0), eb1 = lds8(sc + kr1);
            const uint32_t vb0 = lds8(sc + BN + kr0), vb1 = lds8(sc + BN + kr1);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.k_empty[s]));  // the stage is in registers
            const float f0 = __uint_as_float(eb0 << 23), f1 = __uint_as_float(eb1 << 23);
            p[0][0] = acc[0] * (qs[0] * f0);
            p[0][1] = acc[1] * (qs[1] * f0);
            p[1][0] = acc[2] * (qs[0] * f1);
            p[1][1] = acc[3] * (qs[1] * f1);
            vf[0] = __uint_as_float(vb0 << 23);
            vf[1] = __uint_as_float(vb1 << 23);
            if (__any_sync(0xffffffffu, vb0 == 127u || vb1 == 127u)) {
              if (zero_row<FMT>(a, item, kr0, left, vb0, t)) vf[0] = 0.f;
              if (zero_row<FMT>(a, item, kr1, left, vb1, t)) vf[1] = 0.f;
            }
            // NaN rows (255), and 2^-127, which is no normal number (0).
            if (__any_sync(0xffffffffu, max(max(eb0, eb1), max(vb0 - 1u, vb1 - 1u)) >= 254u)) {
              if (eb0 == 255u) p[0][0] = p[0][1] = NAN;
              if (eb1 == 255u) p[1][0] = p[1][1] = NAN;
              if (vb0 == 255u || vb0 == 0u) vf[0] = vb0 ? NAN : 5.877471754111438e-39f;
              if (vb1 == 255u || vb1 == 0u) vf[1] = vb1 ? NAN : 5.877471754111438e-39f;
              nan_rows = true;
            }
          }
          if (BN > left + min_rel) {  // keys that a row does not see, whatever they hold
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                if ((k ? kr1 : kr0) >= left + rel[n]) p[k][n] = -INFINITY;
            if (kr0 >= left) vf[0] = 0.f;  // (NaN times 0)
            if (kr1 >= left) vf[1] = 0.f;
          }
          bool keep = true;
          if constexpr (LATE) {
            // The rows' maxima over the block: this warp's keys, then all eight warps.
            if (ok) {
              float mt[2];
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                float m = max_nan(p[0][n], p[1][n]);  // (a block with a NaN is not skipped)
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
                mt[n] = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
              }
              if (g == 0) {
                sh.rmax[c & 1][warp][2 * t] = mt[0];
                sh.rmax[c & 1][warp][2 * t + 1] = mt[1];
              }
            }
            named_bar_sync(kVoteBarrier, NCW * 32);
            if (ok) {
              const float c2 = item.x.ln_lam * kLog2e;
              bool vote = true;  // this lane's rows leave the block out
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < NCW; ++w) m = max_nan(m, sh.rmax[c & 1][w][2 * t + n]);
                // With ln(lambda) < 0, "rowmax - m_new < c" is "rowmax - m_old < c".
                const float diff = m == -INFINITY ? -INFINITY : m - m2[n];
                vote = vote && (2 * t + n >= rows || diff < c2 || m == -INFINITY);
                m2[n] = max_nan(m2[n], m);
              }
              keep = !__all_sync(0xffffffffu, vote);  // the same in every warp
              if (tid == 0) {
                const int dc = decided + c;
                if (dc < NDEC || mbar_wait_shared(smem_u32(&sh.dec_empty[dc % NDEC]),
                                                  (dc / NDEC - 1) & 1, abort, a.err)) {
                  sh.dec[dc % NDEC] = keep ? 1 : 0;
                  mbar_arrive(smem_u32(&sh.dec_full[dc % NDEC]));
                }
                if (a.bits) {
                  const uint32_t word = ((c & 31) ? sh.word : 0u) | (keep ? 0u : 1u << (c & 31));
                  sh.word = word;
                  if ((c & 31) == 31 || c == item.x.nb - 1) {
                    const int64_t tile = ((int64_t)item.x.s * a.Hkv + item.hk) * a.n_t + item.x.t;
                    a.bits[(tile * a.n_splits + item.slot) * a.words + (c >> 5)] = word;
                  }
                }
              }
              __syncwarp();
            }
          }
          if (keep && ok) {
            float w[2][2], pv[2][2];
            auto weigh = [&]() {
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  w[k][n] = ex2(p[k][n] - sref[n]);
                  pv[k][n] = w[k][n] * vf[k] * px[n];
                }
            };
            weigh();
            // The references move when a key passes one of them by more than 2^8 (or it
            // is the row's first): then by the warp's maxima.
            const float wm = fmaxf(fmax3(w[0][0], w[1][0], w[0][1]), w[1][1]);
            const float pm = max_nan(max3_nan(pv[0][0], pv[1][0], pv[0][1]), pv[1][1]);
            if (__any_sync(0xffffffffu, wm > 256.f || !(pm <= 32768.f))) {  // 2^8, 2^(8 + 7)
              float al[2];
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                float x = fmaxf(p[0][n], p[1][n]);
                float m = fmaxf(p[0][n] + x_of(vf[0]), p[1][n] + x_of(vf[1]));  // (0 counts as 2^-127)
#pragma unroll
                for (int o = 4; o < 32; o *= 2) {
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                }
                x = fmaxf(sref[n], ceilf(x));
                const float from = sref[n] - x_of(px[n]);  // ref - 7
                const float to = fmaxf(fmaxf(from, ceilf(m) - kPLog2), x - kBelow - kPLog2);
                al[n] = ex2(from - to);
                l[n] *= ex2(sref[n] - x);
                sref[n] = x;
                px[n] = __int_as_float(((int)(x - to) + 127) << 23);
              }
              weigh();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[i][0] *= al[0];
                o[i][1] *= al[1];
                o[i][2] *= al[0];
                o[i][3] *= al[1];
              }
              if constexpr (LATE) {  // the previous block's P, row g of it (a power of two)
                const float even = __shfl_sync(0xffffffffu, al[0], g >> 1);
                const float odd = __shfl_sync(0xffffffffu, al[1], g >> 1), by = (g & 1) ? odd : even;
                b0 = mul_f16x2(b0, pack_f16x2(by, by));
                b1 = mul_f16x2(b1, pack_f16x2(by, by));
              }
            }
            l[0] += w[0][0] + w[1][0];
            l[1] += w[0][1] + w[1][1];
            if (nan_rows) {  // (they do not reach the rows that they are hidden from)
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                  if (p[k][n] == -INFINITY) pv[k][n] = 0.f;
            }
            // P as the B operand: key pairs of row g.
            n0 = transpose8x8(pack_f16x2(pv[0][0], pv[0][1]));
            n1 = transpose8x8(pack_f16x2(pv[1][0], pv[1][1]));
            fresh = true;
          }
        }
        if constexpr (!LATE) {
          pending = fresh;
          b0 = n0;
          b1 = n1;
        }
        if (pending && ok) {
          const int vs = vn < NST ? vn : vn - NST;
          ok = wait_warp(&sh.v_full[vs], vn >= NST);
          const int vleft = LATE ? left + BN : left;  // its block's rows below kv
          const uint32_t vt = base + L::V + vs * L::CODES;
          if constexpr (FMT == kKvE4m3) {
            uint4 r0 = lds128(chunk_at<FMT>(vt, vr0, g)), r1 = lds128(chunk_at<FMT>(vt, vr1, g));
            uint4 r2 = lds128(chunk_at<FMT>(vt, vr0 + 8, g)), r3 = lds128(chunk_at<FMT>(vt, vr1 + 8, g));
            if (vleft < BN) {  // rows at or past kv may hold anything
              if (vr0 >= vleft) r0 = make_uint4(0, 0, 0, 0);
              if (vr1 >= vleft) r1 = make_uint4(0, 0, 0, 0);
              if (vr0 + 8 >= vleft) r2 = make_uint4(0, 0, 0, 0);
              if (vr1 + 8 >= vleft) r3 = make_uint4(0, 0, 0, 0);
            }
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
            const uint32_t w2[4] = {r2.x, r2.y, r2.z, r2.w}, w3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // four dims: two m-tiles
              uint32_t a0, a1, a2, a3;
              e4m3x4(__byte_perm(w0[i], w1[i], 0x5140), a0, a1);
              e4m3x4(__byte_perm(w2[i], w3[i], 0x5140), a2, a3);
              mma16816(o[2 * i], a0, a1, a2, a3, b0, b1);
              e4m3x4(__byte_perm(w0[i], w1[i], 0x7362), a0, a1);
              e4m3x4(__byte_perm(w2[i], w3[i], 0x7362), a2, a3);
              mma16816(o[2 * i + 1], a0, a1, a2, a3, b0, b1);
            }
          } else {
            // The lane's sixteen dims are one block: eight bytes of half a chunk.
            auto row8 = [&](int r) { return lds64(chunk_at<FMT>(vt, r, g >> 1) + (g & 1) * 8); };
            const uint32_t vx = base + L::VX + vs * C::BS;
            uint2 r0 = row8(vr0), r1 = row8(vr1), r2 = row8(vr0 + 8), r3 = row8(vr1 + 8);
            uint32_t e0 = lds8(vx + vr0 * 8 + g), e1 = lds8(vx + vr1 * 8 + g);
            uint32_t e2 = lds8(vx + (vr0 + 8) * 8 + g), e3 = lds8(vx + (vr1 + 8) * 8 + g);
            if (vleft < BN) {
              if (vr0 >= vleft) r0 = make_uint2(0, 0), e0 = 0;
              if (vr1 >= vleft) r1 = make_uint2(0, 0), e1 = 0;
              if (vr0 + 8 >= vleft) r2 = make_uint2(0, 0), e2 = 0;
              if (vr1 + 8 >= vleft) r3 = make_uint2(0, 0), e3 = 0;
            }
            uint32_t s01, s23;
            e4m3x4(e0 | (e1 << 8) | (e2 << 16) | (e3 << 24), s01, s23);
            const uint32_t w0[2] = {r0.x, r0.y}, w1[2] = {r1.x, r1.y}, w2[2] = {r2.x, r2.y},
                           w3[2] = {r3.x, r3.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // eight dims: four m-tiles
              // A byte of a row is dims (2 k, 2 k + 1); a pair byte needs the same dim of
              // two keys: even dims of both, then odd dims of both.
              const uint32_t ev01 = (w0[i] & 0x0f0f0f0fu) | ((w1[i] & 0x0f0f0f0fu) << 4);
              const uint32_t od01 = ((w0[i] >> 4) & 0x0f0f0f0fu) | (w1[i] & 0xf0f0f0f0u);
              const uint32_t ev23 = (w2[i] & 0x0f0f0f0fu) | ((w3[i] & 0x0f0f0f0fu) << 4);
              const uint32_t od23 = ((w2[i] >> 4) & 0x0f0f0f0fu) | (w3[i] & 0xf0f0f0f0u);
              uint32_t x0[4], x1[4], x2[4], x3[4];
              e2m1x8(ev01, x0);
              e2m1x8(od01, x1);
              e2m1x8(ev23, x2);
              e2m1x8(od23, x3);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma16816(o[4 * i + k], mul_f16x2(x0[k], s01), mul_f16x2(x1[k], s01),
                         mul_f16x2(x2[k], s23), mul_f16x2(x3[k], s23), b0, b1);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.v_empty[vs]));
          vn = vn == 2 * NST - 1 ? 0 : vn + 1;
        }
        if constexpr (LATE) {
          pending = fresh;
          b0 = n0;
          b1 = n1;
        }
      }
    };
    if (dense)
      blocks(std::false_type{});
    else
      blocks(std::true_type{});

    // ---- merge of the eight warps: O = sum_w 2^(ref_w - S - 7) O_w / L, L = sum_w
    // 2^(sref_w - S) l_w, S the largest sref ----------------------------------------
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 4);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 8);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 16);
    }
    // Every warp is here: the merge area's last readers have left it.
    if (bar_red_or(kVoteBarrier, NCW * 32, !ok)) return;
    if (g == 0) {
      sh.ml[0][warp][2 * t] = sref[0] - x_of(px[0]);
      sh.ml[0][warp][2 * t + 1] = sref[1] - x_of(px[1]);
      sh.ml[1][warp][2 * t] = l[0];
      sh.ml[1][warp][2 * t + 1] = l[1];
      sh.ml[2][warp][2 * t] = sref[0];
      sh.ml[2][warp][2 * t + 1] = sref[1];
    }
    // Warp r sums row r of the warps' outputs, COLS columns at a time: PER of every
    // sixteen.  A CTA with one tile has the code tiles to do it in, at once; where
    // others follow, their keys and values are on the way there.
    auto merge = [&](auto columns, float *area) {
      constexpr int COLS = decltype(columns)::value, PER = COLS / 8, VEC = COLS / 32, STRIDE = COLS + 4;
      const int r = warp;
      const int64_t orow = (int64_t)(x.tok0 + r / a.G) * a.Hq + item.hk * a.G + r % a.G;
      float f[NCW], iz = 0.f;
#pragma unroll
      for (int q = 0; q < D / COLS; ++q) {
        if (q) named_bar_sync(kVoteBarrier, NCW * 32);
        float *at = area + (warp * ROWS + 2 * t) * STRIDE + PER * g;
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const int m = (q * PER + 4 * i) / 2;
          *reinterpret_cast<float4 *>(at + 4 * i) =
              make_float4(o[m][0], o[m][2], o[m + 1][0], o[m + 1][2]);
          *reinterpret_cast<float4 *>(at + STRIDE + 4 * i) =
              make_float4(o[m][1], o[m][3], o[m + 1][1], o[m + 1][3]);
        }
        named_bar_sync(kVoteBarrier, NCW * 32);
        if (r >= rows) continue;
        if (q == 0) {
          float m = -INFINITY, y = -INFINITY, z = 0.f;
#pragma unroll
          for (int w = 0; w < NCW; ++w)
            if (sh.ml[1][w][r] != 0.f) {
              m = fmaxf(m, sh.ml[2][w][r]);
              y = fmaxf(y, sh.ml[0][w][r]);
            }
#pragma unroll
          for (int w = 0; w < NCW; ++w) {
            const float lw = sh.ml[1][w][r];
            f[w] = lw == 0.f ? 0.f : ex2(sh.ml[0][w][r] - y);  // 0: the warp met no key of the row
            if (lw != 0.f) z = fmaf(lw, ex2(sh.ml[2][w][r] - m), z);
          }
          iz = z == 0.f ? 0.f : ex2(y - m) / z;
          if (lane == 0)
            (a.n_splits == 1 ? a.lse : a.lse_part)[orow * a.n_splits + item.slot] =
                z == 0.f ? -INFINITY : m * kLn2 + logf(z);
          // Slots behind the tile's last partial have no weight.
          for (int i = item.slot + 1 + lane; i < item.fill; i += 32)
            a.lse_part[orow * a.n_splits + i] = -INFINITY;
        }
        const int pos = lane * VEC, d = 16 * (pos / PER) + q * PER + pos % PER;
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < NCW; ++w) {
          const float *u = area + (w * ROWS + r) * STRIDE + pos;
          if constexpr (VEC == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(u);
            v[0] = fmaf(y.x, f[w], v[0]);
            v[1] = fmaf(y.y, f[w], v[1]);
            v[2] = fmaf(y.z, f[w], v[2]);
            v[3] = fmaf(y.w, f[w], v[3]);
          } else {
            v[0] = fmaf(*u, f[w], v[0]);
          }
        }
        __nv_bfloat16 *out = (__nv_bfloat16 *)a.o + orow * D + d;
        float *part = a.o_part + (orow * a.n_splits + item.slot) * D + d;
        if constexpr (VEC == 4) {
          if (a.n_splits == 1)
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(pack_bf16x2(v[0] * iz, v[1] * iz), pack_bf16x2(v[2] * iz, v[3] * iz));
          else
            *reinterpret_cast<float4 *>(part) = make_float4(v[0] * iz, v[1] * iz, v[2] * iz, v[3] * iz);
        } else {
          *part = v[0] * iz;  // (more than one split)
        }
      }
    };
    if (a.shared_out)
      merge(std::integral_constant<int, MERGE_COLS>{}, reinterpret_cast<float *>(smem_raw + L::MERGE));
    else
      merge(std::integral_constant<int, D>{}, reinterpret_cast<float *>(smem_raw));
    if (!dense) decided += item.x.nb;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[it & 1]));
  }
}

// 4-D map over the code rows of a page pool: (byte, slot, head, page).
bool make_map_codes(CUtensorMap *m, const KvPages &p, const void *ptr, int row) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)row, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv,
                              (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)row, (cuuint64_t)p.page_size * row,
                                 (cuuint64_t)p.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)row, (cuuint32_t)(p.page_size < BN ? p.page_size : BN), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
cudaError_t launch_fmt(const ChunkArgs &a, unsigned grid, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!make_map_codes(&mk, a.pages, a.pages.k, Cfg<FMT>::ROW) ||
      !make_map_codes(&mv, a.pages, a.pages.v, Cfg<FMT>::ROW))
    return cudaErrorInvalidValue;
  constexpr uint32_t smem = Layout<FMT>::END + ((sizeof(Shared) + 15) / 16) * 16;
  const cudaError_t e = cudaFuncSetAttribute(decode_paged_kernel<FMT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode_paged_kernel<FMT><<<grid, NT, smem, s>>>(mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_paged(const ChunkArgs &args, unsigned grid, cudaStream_t s) {
  ChunkArgs a = args;
  // More pieces than CTAs fit: shared out on the device, up to 128 sequences (with
  // more of them a CTA's search through the list costs what it saves).
  const int64_t list = (int64_t)a.n_seq * a.Hkv * ((a.max_kv + BN - 1) / BN);
  if (grid > kCtas && a.n_splits > 1 && a.n_seq <= 32 * SEQS && list > 0 && list < (int64_t)1 << 30) {
    a.shared_out = 1;
    grid = kCtas;
  }
  return a.pages.format == kKvE4m3 ? launch_fmt<kKvE4m3>(a, grid, s) : launch_fmt<kKvNvfp4>(a, grid, s);
}

}  // namespace attn_skip
