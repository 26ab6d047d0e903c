// Attention of a chunk of new tokens over a paged key/value cache, with
// softmax-threshold block skipping (d = 128, 128-key blocks), on tcgen05.
//
// Method: the BLASST page, sections "BLASST 的判定准则" (Eq. 5), "Prefill 内核：
// 砍计算" and "Decode 内核：砍带宽"; the loop is that of the prefill kernel.  With
// i a token of a sequence's chunk of n tokens and kv the sequence's cached
// length (chunk included), query (i, head) sits at position p = kv - n + i and
//     s_c = scale <q, k_c>,   c < kv,   causal: c <= p
//     O = sum_c exp(s_c - LSE) v_c,   LSE = ln sum_c exp(s_c)   (kept blocks)
//
// One CTA per (tile, KV head, split).  A tile is TT = floor(128 / G)
// consecutive tokens times the G query heads that share the KV head, so the
// 128 rows of the products are full for chunks of any length above 128 / G and
// every key is read once for G heads (a tile of one head's 128 tokens would
// leave a decode step 1 row of 128).  Row r is token r / G, head r % G: one
// TMA box of G heads x TT tokens.  A split owns bps blocks of the key axis and
// restarts its running max; with more than one split the partial outputs are
// merged by log-sum-exp in a second launch.  Many short tiles over bf16 rows run in
// CTAs that stay (prompt_paged_kernel, below), tiles of at most eight rows over a
// quantised cache on warp-level products (decode_paged.cu).
//
// Warp roles:
//   0-3   deciders: row max of S_j, vote against the running max, AND;
//   4-7   exponentials: P_j = exp2(S_j - ref) into TMEM, row sums, O rescale;
//   8     key producer: page ids, then one copy per page (or part of a page);
//   9     Q.K^T issuer; a bf16 cache has two (9, 12: even / odd blocks), since a
//         thread that issues tcgen05.mma is held until the tensor pipe takes
//         each instruction;
//   10    value producer, kept blocks only;
//   11    P.V issuer;
//   12-15, 16-19 (E4M3 and NVFP4 caches) key and value converters: codes from
//         a staging ring to fp16 tiles in the layout that TMA gives a bf16
//         cache; before that, Q to fp16.
//
// Quantised caches.  cvt widens two codes to fp16 in one instruction, at the
// rate of any other; a bf16 pair takes five.  fp16's range is met by exponents
// that cost nothing per score: with E_k and E_v the largest row-scale exponents
// of a block's keys and values, the tiles hold code * 2^(e - E) (exact for e >=
// E - 15, otherwise off by at most 2^-25 2^E; NVFP4, whose block scale takes the
// factor first, 7 times that), the scores of the block are
// scaled by 2^E_k, and P takes 2^E_v: with sref the running max of the row maxima and
// ref that of (row max + E_v), both of which may lag by 2^8,
//     P'_c = 2^(s_c - sref + f),  f = sref + E_v - ref + 7,  l += 2^-f sum P'_c.
// P' stays below fp16's 2^16, has its 11 bits down to 2^-21 of the largest contribution
// and steps of 2^-31 of it below (it counts where the row with the large weight
// holds a zero).  f is -40 at least, where P' is 0 in fp16, so that the weights stay
// in fp32's range: the values' exponents span as much, and without a reference on
// the scores alone the weights of blocks of small values were lost beside blocks of
// large ones.  A block whose values are all zero (E_v = -inf) has no part in ref.
// A query row enters as fp16(q * 2^x), 2^x the largest power of two with max|q| 2^x
// <= 2^15.
//
// A warp quarter whose 32 rows lie past the tile's last row (decode: G rows) has
// no decider and no exponential warp: they convert, or go to the end at once.
//
// Tiles of at most 32 rows (decode, drafted tokens) stand in all four quarters of
// the 128 product rows: quarter w exponentiates keys 32 w .. 32 w + 31 of each
// block against its own running reference, its P holding zeros for the other
// keys, and the four partial outputs are merged as splits are.  One warp with
// all 128 keys of a handful of rows was what bounded decode over the quantised
// caches (3600 cycles a block on an SM whose other warps convert).
//
// Rows of the last block at or past the last key that some row of the tile sees
// (later tokens, a page's unwritten tail, pages never loaded) may hold anything:
// their scores are replaced by -inf, and their values are left out of the product:
// over bf16 rows P.V goes over whole sixteens of keys, up to the one with the last
// such key, and the value rows behind that key become zeros in shared memory;
// converters write zeros for all of them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace attn_skip {
namespace {

using namespace tc;

constexpr int BM = 128;   // rows of a tile
constexpr int NR = 4;     // barrier ring of the blocks (even, and longer than NS)
constexpr int NV = 2;     // bf16 value tiles
constexpr int NS = 3;     // TMEM S buffers
constexpr int NDEC = 4;   // decision ring
constexpr int NE = 8;     // scale exponent ring of the quantised formats
constexpr int NQ = 4;     // warps per row role
constexpr int kDeciderBarrier = 1, kMergeBarrier = 2;
constexpr int MERGE_STRIDE = D + 4;  // floats a row: a row's 16-byte stores meet other banks than the next's
constexpr int WARP_K = 8, WARP_MMA = 9, WARP_V = 10, WARP_PV = 11;
constexpr int WARP_MMA2 = 12;             // bf16 cache
constexpr int WARP_KC = 12, WARP_VC = 16;  // quantised caches
constexpr uint32_t TILE_BYTES = BM * D * 2;
constexpr uint32_t HALF_BYTES = TILE_BYTES / 2;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_O = NS * BN;
constexpr uint32_t IDESC_QK = idesc_bf16_f32(BM, BN, 0);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(BM, D, 1);
constexpr uint32_t IDESC_QK16 = idesc_f16_f32(BM, BN, 0);
constexpr uint32_t IDESC_PV16 = idesc_f16_f32(BM, D, 1);
constexpr uint32_t NEG_INF_BITS = 0xff800000u;

// Per format: bf16 key tiles (NKD), the staging rings of the quantised formats
// (NC stages each for keys and values) and what a staged block holds.
template <int FMT> struct Cfg;
template <> struct Cfg<kKvBf16> {
  static constexpr int NKD = 4, NC = 0, WARPS = 13;
  static constexpr uint32_t ROW = 2 * D, CODES = 0, BS = 0;
};
template <> struct Cfg<kKvE4m3> {
  static constexpr int NKD = 2, NC = 2, WARPS = 20;
  static constexpr uint32_t ROW = D, CODES = BN * D, BS = 0;
};
template <> struct Cfg<kKvNvfp4> {
  static constexpr int NKD = 2, NC = 3, WARPS = 20;
  static constexpr uint32_t ROW = D / 2, CODES = BN * D / 2, BS = BN * D / 16;
};
// PAIR: two CTAs an SM, one tile each for keys and values.
template <int FMT, bool PAIR = false> struct Layout {
  using C = Cfg<FMT>;
  static constexpr int NKD = PAIR ? 1 : C::NKD, NV = PAIR ? 1 : attn_skip::NV;
  static constexpr uint32_t Q = 0, K = TILE_BYTES, V = K + NKD * TILE_BYTES;
  // A staged block: codes, block scales, row scales; a key block's stage also
  // holds the row scales of its values (needed before the values are).
  static constexpr uint32_t SCALES = C::CODES + C::BS, KSTAGE = SCALES + 2 * BN, VSTAGE = SCALES + BN;
  static constexpr uint32_t KC = V + NV * TILE_BYTES, VC = KC + C::NC * KSTAGE;
  static constexpr uint32_t END = VC + C::NC * VSTAGE;
};

struct Shared {
  uint64_t q_full;
  uint64_t ready[NR];    // slot c % NR: block c's key tile is in and its S buffer free
  uint64_t qk_done[NR];  // slot c % NR: block c's Q.K^T complete
  uint64_t v_full[NV], v_empty[NV];
  uint64_t p_full[NS], pv_done[NS];
  uint64_t dec_full[NDEC], dec_read[NDEC];
  uint64_t l_full;
  uint64_t v_tail;       // the last block's value rows, before their tail is zeroed
  uint64_t kc_full[3], kc_empty[3], vc_full[3], vc_empty[3];
  uint64_t q_ready;      // Q as fp16
  int dec[NDEC];
  // Scale bytes (E_k, E_v; 0 where all values are) of block c, slot c % NE.  Slot
  // reuse: block c + NE is converted after block c + NE - NKD's Q.K^T, whose S buffer was block c +
  // NE - NKD - NS's (NE - NKD - NS > 0), by then read by everyone.
  uint16_t esc[NE];
  int8_t qexp[BM];       // x of the query rows
  // [S buffer][row] running max after the buffer's block (log2 units; a quantised
  // cache: the block's maximum).  Row sums and exp references (sref, ref) for the
  // epilogue take the buffers' place at the end: row r's words are read and written
  // by its two threads alone.
  // REP: the exponential warps take the maximum themselves, and the last buffer
  // holds the row maxima of the quarters' keys.
  float mdec[NS][BM];
  TileInfo tile;
  uint32_t tmem_base;
  int abort;
};
static_assert(Layout<kKvBf16>::END + sizeof(Shared) <= 227 * 1024, "shared memory budget");
static_assert(Layout<kKvE4m3>::END + sizeof(Shared) <= 227 * 1024, "shared memory budget");
static_assert(Layout<kKvNvfp4>::END + sizeof(Shared) <= 227 * 1024, "shared memory budget");
static_assert(2 * (Layout<kKvBf16, true>::END + sizeof(Shared) + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(NQ * 32 * MERGE_STRIDE * 4 <= 3 * TILE_BYTES, "merge area: query, key and value tiles");
static_assert(NR % 2 == 0 && NR > NS, "barrier ring: even, and longer than the S buffer ring");

__device__ __forceinline__ uint64_t kmajor_base(uint32_t tile) {
  return smem_desc_sw128(tile, 16u, 1024u);
}
__device__ __forceinline__ constexpr uint64_t kmajor_step(int kk) {
  return (uint64_t)(((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4);
}
__device__ __forceinline__ uint64_t vmajor_base(uint32_t tile) {
  return smem_desc_sw128(tile, HALF_BYTES, 1024u);
}
__device__ __forceinline__ constexpr uint64_t vmajor_step(int kk) {
  return (uint64_t)(((uint32_t)kk * 2048u) >> 4);
}

// O (+)= P V over the sixteens of a block's keys with one below `left`: the last
// block's, out of line, and whole blocks'.  (A test before every instruction costs
// the issuer 6 % of a chunk of 4096 on 16384.)
__device__ __noinline__ void issue_pv_part(uint32_t o, uint32_t p, uint64_t v, uint32_t idesc, uint32_t add,
                                           int left) {
#pragma unroll 1
  for (int kk = 0; kk * 16 < left; ++kk)
    mma_bf16_ts(o, p + kk * 8, v + vmajor_step(kk), idesc, kk > 0 ? 1u : add);
}
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint64_t v, uint32_t idesc, bool add,
                                         int left) {
  if (left >= BN) {
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk)
      mma_bf16_ts(o, p + kk * 8, v + vmajor_step(kk), idesc, kk > 0 || add ? 1u : 0u);
  } else {
    issue_pv_part(o, p, v, idesc, add ? 1u : 0u, left);
  }
}

// Of 32 * chunks keys, those at or past the row's `left` become -inf in this
// warp's TMEM lanes; 32 keys at a time, chunks without a hidden key are left
// alone.
__device__ __noinline__ void mask_block_tmem(uint32_t sa, int left, int chunks) {
  uint32_t ninf[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) ninf[i] = NEG_INF_BITS;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const int lim = left - 32 * c;
    if (__all_sync(0xffffffffu, lim >= 32)) continue;
    if (__all_sync(0xffffffffu, lim <= 0)) {
      tmem_st32(sa + 32 * c, ninf);
      continue;
    }
    uint32_t x[32];
    tmem_ld32(sa + 32 * c, x);
    tmem_wait_ld_regs(x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i < lim ? x[i] : NEG_INF_BITS;
    tmem_st32(sa + 32 * c, x);
  }
  tmem_wait_st();
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A NaN among the scores is their maximum: a block that holds one is not skipped.
__device__ __forceinline__ float chunk_max(const uint32_t (&s)[32]) {
  float m[11];
#pragma unroll
  for (int i = 0; i < 10; ++i)
    m[i] = max3_nan(__uint_as_float(s[3 * i]), __uint_as_float(s[3 * i + 1]),
                    __uint_as_float(s[3 * i + 2]));
  m[10] = max_nan(__uint_as_float(s[30]), __uint_as_float(s[31]));
  const float a = max3_nan(m[0], m[1], m[2]), b = max3_nan(m[3], m[4], m[5]);
  const float c = max3_nan(m[6], m[7], m[8]), d = max_nan(m[9], m[10]);
  return max_nan(max3_nan(a, b, c), d);
}

// P = exp2(s * sl2 - ref) for 32 keys as 16 packed bf16 (fp16) pairs, the P.V
// product's operand type; the row sum takes the unrounded fp32 values.
template <bool F16>
__device__ __forceinline__ void chunk_exp(const uint32_t (&s)[32], uint64_t sl2x2,
                                          uint64_t negref2, uint64_t (&acc)[2], uint32_t *pk) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    f2_split(f2_fma(f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sl2x2,
                    negref2),
             x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    acc[i & 1] = f2_add(acc[i & 1], f2(p0, p1));
    pk[i] = F16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
  }
}

// Block j's rows (codes and scales) into the staging area or tile at dst, part by
// part, one lane a part; whole warp.  The arrival with the byte count comes
// first.
template <int FMT>
__device__ __forceinline__ void load_block_here(const ChunkArgs &a, Producer &p, const CUtensorMap *map,
                                        bool value, int j, uint32_t dst, uint32_t full, int lane) {
  using C = Cfg<FMT>;
  constexpr bool QUANT = FMT != kKvBf16;
  const int sub = 1 << p.lsub;
  const Part x = part_of(a, p, j, lane);
  const int n = x.n, page = x.page, slot = x.slot;
  if (lane == 0) mbar_expect_tx(full, n * sub * (C::ROW + (QUANT ? (value ? 1 : 2) + C::BS / BN : 0)));
  __syncwarp();
  if (lane < n) {
    if constexpr (!QUANT) {
      const uint32_t d = dst + lane * sub * 128;
      tma_load_4d(d, map, full, 0, slot, p.hk, page, p.policy);
      tma_load_4d(d + HALF_BYTES, map, full, 64, slot, p.hk, page, p.policy);
    } else {
      const KvPages &g = a.pages;
      const int64_t row = ((int64_t)page * g.Hkv + p.hk) * g.page_size + slot;
      const uint8_t *src = (const uint8_t *)(value ? g.v : g.k) + (int64_t)page * g.page_stride +
                           ((int64_t)p.hk * g.page_size + slot) * C::ROW;
      const uint32_t r0 = lane * sub, scales = dst + Layout<FMT>::SCALES + r0;
      bulk_load(dst + r0 * C::ROW, src, sub * C::ROW, full, p.policy);
      if constexpr (FMT == kKvNvfp4)
        bulk_load(dst + C::CODES + r0 * (D / 16), (value ? g.v_bs : g.k_bs) + row * (D / 16),
                  sub * (D / 16), full, p.policy);
      bulk_load(scales, (value ? g.v_scale : g.k_scale) + row, sub, full, p.policy);
      if (!value) bulk_load(scales + BN, g.v_scale + row, sub, full, p.policy);
    }
  }
  __syncwarp();
}

// Out of line for the quantised formats, whose converters need the instruction
// cache; in line for bf16 (decode of 16 x 32768: 339 against 322 us).
template <int FMT>
__device__ __noinline__ void load_block_call(const ChunkArgs &a, Producer &p, const CUtensorMap *map,
                                             bool value, int j, uint32_t dst, uint32_t full,
                                             int lane) {
  load_block_here<FMT>(a, p, map, value, j, dst, full, lane);
}
template <int FMT>
__device__ __forceinline__ void load_block(const ChunkArgs &a, Producer &p, const CUtensorMap *map,
                                           bool value, int j, uint32_t dst, uint32_t full,
                                           int lane) {
  if constexpr (FMT == kKvBf16)
    load_block_here<FMT>(a, p, map, value, j, dst, full, lane);
  else
    load_block_call<FMT>(a, p, map, value, j, dst, full, lane);
}

// ------------------------------------------------------------- conversions --
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Four E4M3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Eight E2M1 codes (element 2i in byte i's low nibble) as four fp16 pairs (exact).
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// fp16 pair of 2^(byte - top): 1 for a row of zeros above the block's top, 0
// below 2^-24, NaN for byte 255.
__device__ __forceinline__ uint32_t row_factor(int byte, int top) {
  const int r = min(byte - top, 0);
  uint32_t f = r >= -14 ? (uint32_t)(r + 15) << 10 : r >= -24 ? 1u << (r + 24) : 0u;
  if (byte == 255) f = 0x7e00u;
  return f | (f << 16);
}

// The largest scale byte of a block's rows below `left`; whole warp, lane l
// brings the bytes of rows 4 l .. 4 l + 3.  Rows of byte 255 (NaN) do not count,
// nor rows of zeros, which the writer gives byte 127: where that is the largest
// byte, the codes are looked up in the cache (not in the staging area: a block's
// values come after its scales).  0 for zeros alone.
template <int FMT>
__device__ __noinline__ int block_top_slow(const ChunkArgs &a, const TileInfo &x, int hk, int j,
                                           bool value, const uint8_t *scales, int lane, int left) {
  const KvPages &p = a.pages;
  int top = 0;
  bool nan = false;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * lane + i;
    if (r < left && scales[r] == 255) nan = true;
    if (r >= left || scales[r] == 255) continue;
    uint32_t any = 1;
    if (scales[r] == 127) {
      const int pos = j * BN + r;
      int page = __ldg(a.page_table + (int64_t)x.s * a.max_pages + pos / p.page_size);
      if (page < 0 || page >= p.n_pages) page = 0;
      const uint4 *c = reinterpret_cast<const uint4 *>(
          (const uint8_t *)(value ? p.v : p.k) + page * p.page_stride +
          ((int64_t)hk * p.page_size + pos % p.page_size) * Cfg<FMT>::ROW);
      any = 0;
      for (uint32_t k = 0; k < Cfg<FMT>::ROW / 16; ++k) {
        const uint4 w = __ldg(c + k);
        any |= w.x | w.y | w.z | w.w;
      }
      any &= FMT == kKvE4m3 ? 0x7f7f7f7fu : 0x77777777u;
    }
    if (any) top = max(top, (int)scales[r]);
  }
  top = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
  return top || !__any_sync(0xffffffffu, nan) ? top : 127;
}

template <int FMT>
__device__ __forceinline__ int block_top(const ChunkArgs &a, const TileInfo &x, int hk, int j,
                                         bool value, const uint8_t *scales, int lane) {
  uint32_t w = reinterpret_cast<const uint32_t *>(scales)[lane];
  const int left = x.kv - j * BN;  // rows of the block that count
  if (left < BN) {
    const int mine = left - 4 * lane;
    w &= mine >= 4 ? 0xffffffffu : mine <= 0 ? 0u : (1u << (8 * mine)) - 1u;
  }
  const uint32_t m = __vmaxu2(w & 0x00ff00ffu, (w >> 8) & 0x00ff00ffu);
  const int top = (int)__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if (top != 255 && top != 127 && top != 0) return top;
  return block_top_slow<FMT>(a, x, hk, j, value, scales, lane, left);
}

// Step g of a staged block to an fp16 tile: rows 4 g .. 4 g + 3, eight lanes a
// row, sixteen codes each.  Lanes of the upper half of a row store their two
// 16-byte chunks in the other order, so that a store instruction's eight lanes
// of a row meet eight different bank groups.
template <int FMT> struct Step {
  uint4 c;
  uint32_t b, byte;

  __device__ __forceinline__ void load(const uint8_t *stage, int g, int lane) {
    const int r = g * 4 + (lane >> 3), cg = lane & 7;
    byte = stage[Layout<FMT>::SCALES + r];
    if constexpr (FMT == kKvE4m3) {
      c = *reinterpret_cast<const uint4 *>(stage + r * D + cg * 16);
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(stage + r * (D / 2) + cg * 8);
      c.x = v.x;
      c.y = v.y;
      b = stage[Cfg<FMT>::CODES + r * (D / 16) + cg];
    }
  }
  __device__ __forceinline__ void store(uint32_t tile, int g, int lane, int top, int rows_left) {
    const int rl = lane >> 3, cg = lane & 7;
    const bool upper = cg >= 4;
    uint32_t f = row_factor(byte, top);
    uint32_t h[8];
    if constexpr (FMT == kKvE4m3) {
      e4m3x4(c.x, h[0], h[1]);
      e4m3x4(c.y, h[2], h[3]);
      e4m3x4(c.z, h[4], h[5]);
      e4m3x4(c.w, h[6], h[7]);
    } else {
      uint32_t s0, s1;
      e2m1x8(c.x, *reinterpret_cast<uint32_t(*)[4]>(&h[0]));
      e2m1x8(c.y, *reinterpret_cast<uint32_t(*)[4]>(&h[4]));
      e4m3x4(b * 0x101u, s0, s1);  // the block scale as a pair
      f = mul_f16x2(s0, f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = mul_f16x2(h[k], f);
    if (rows_left < BN && g * 4 + rl >= rows_left) {
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = 0u;
    }
    // Chunk c of row r sits at c ^ (r % 8); the lane's pair is 2 cg % 8 and the next.
    const uint32_t row = tile + (upper ? HALF_BYTES : 0) + (g * 4 + rl) * 128;
    const uint32_t a0 = row + ((((2 * cg) & 7) ^ ((g & 1) * 4 + rl)) * 16), a1 = a0 ^ 16u;
    if (!upper) {
      st_shared_v4(a0, h[0], h[1], h[2], h[3]);
      st_shared_v4(a1, h[4], h[5], h[6], h[7]);
    } else {
      st_shared_v4(a1, h[4], h[5], h[6], h[7]);
      st_shared_v4(a0, h[0], h[1], h[2], h[3]);
    }
  }
};

// Warp w of n takes steps w, w + n, ..; two at a time, their codes read before
// the first store (a store orders every later load behind it).  The steps are a
// loop: twenty warps in eight roles share the instruction cache, and unrolled
// they ran three times slower, at its refill rate.
// rows_left: rows at or past it become zero (values of the last block).
template <int FMT>
__device__ __forceinline__ void convert_block(const uint8_t *stage, uint32_t tile, int w, int n,
                                              int lane, int top, int rows_left) {
#pragma unroll 1
  for (int g = w; g < BN / 4; g += 2 * n) {
    Step<FMT> s, t;
    s.load(stage, g, lane);
    const bool two = g + n < BN / 4;
    if (two) t.load(stage, g + n, lane);
    s.store(tile, g, lane, top, rows_left);
    if (two) t.store(tile, g + n, lane, top, rows_left);
  }
}

// Query rows [r0, r1) of the swizzled bf16 tile to fp16, in place: sixteen lanes
// a row, one 16-byte chunk each.
__device__ __forceinline__ void convert_q(uint32_t tile, int r0, int r1, int lane, int8_t *qexp) {
  for (int r = r0 + (lane >> 4); r < ((r1 + 1) & ~1); r += 2) {
    const uint32_t at = tile + ((lane & 8) ? HALF_BYTES : 0) + r * 128 + (lane & 7) * 16;
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
    float x[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
      m = fmaxf(m, isfinite(x[i]) ? fabsf(x[i]) : 0.f);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int b = __float_as_int(m);
    int e = 15 + 127 - (b >> 23) - ((b & 0x7fffff) != 0 ? 1 : 0);
    e = m > 0.f ? min(e, 100) : 0;
    const float f = __int_as_float((e + 127) << 23);  // e in [-113, 100]
    st_shared_v4(at, pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f),
                 pack_f16x2(x[4] * f, x[5] * f), pack_f16x2(x[6] * f, x[7] * f));
    if ((lane & 15) == 0) qexp[r] = (int8_t)e;
  }
}

// REP: tiles of at most 32 rows, once in each quarter of the products' 128 rows.
// PAIR (REP): in half an SM, for splits of few blocks, whose set-up and last steps
// then lie under another CTA's loads.
template <int FMT, bool REP, bool PAIR>
__global__ void __launch_bounds__(Cfg<FMT>::WARPS * 32, PAIR ? 2 : 1)
    chunk_paged_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ ChunkArgs a, const int q_box_tokens) {
  using C = Cfg<FMT>;
  using L = Layout<FMT, PAIR>;
  constexpr bool QUANT = FMT != kKvBf16;
  constexpr int NKD = L::NKD, NV = L::NV, NC = QUANT ? C::NC : 1;
  constexpr int NS = PAIR ? 1 : attn_skip::NS;
  constexpr uint32_t TMEM_O = NS * BN, TMEM_COLS = PAIR ? 256 : attn_skip::TMEM_COLS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw + L::END);
  const uint32_t base = smem_u32(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (base & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (tid == 0) atomicOr(a.err, kErrLayout);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits for this grid's end)
  const int sp = (int)(blockIdx.x % a.n_splits);
  const int hk = (int)(blockIdx.x / a.n_splits) % a.Hkv;
  const int ti = (int)(blockIdx.x / a.n_splits / a.Hkv);
  volatile int *abort = &sh.abort;
  auto bar = [&](uint64_t *b) { return smem_u32(b); };
  auto wait = [&](uint64_t *b, int phase) {
    return mbar_wait_shared(smem_u32(b), phase & 1, abort, a.err);
  };
  auto wait_warp = [&](uint64_t *b, int phase) {
    return __all_sync(0xffffffffu, mbar_wait_shared(smem_u32(b), phase & 1, abort, a.err));
  };

  Producer pages;  // of the two producer warps
  auto k_dst = [&](int c) { return QUANT ? base + L::KC + (c % NC) * L::KSTAGE : base + L::K + (c % NKD) * TILE_BYTES; };
  auto k_bar = [&](int c) { return QUANT ? &sh.kc_full[c % NC] : &sh.ready[c % NR]; };
  auto load_k = [&](int c) {
    load_block<FMT>(a, pages, &tm_k, false, sh.tile.j0 + c, k_dst(c), bar(k_bar(c)), lane);
  };

  // Set-up: the producers find the tile and its first pages; meanwhile other warps
  // initialise the barriers and allocate TMEM.
  constexpr int K_AHEAD = QUANT ? NC : NKD;  // key blocks that the ring holds
  if (warp == WARP_K || warp == WARP_V) {
    const TileInfo t = producer_tile(a, pages, ti, sp, hk, lane);
    if (warp == WARP_K && lane == 0) {
      sh.tile = t;
      // Readers of a decision: the P.V issuer and the exponential warps that have
      // rows; with a threshold also the value producer and converters.
      const int nq = REP ? NQ : (t.ntok * a.G + 31) / 32, nc = 8 - nq;  // see below
      const int readers = 1 + nq + (t.ln_lam == -INFINITY ? 0 : QUANT ? 1 + nc : 1);
      for (int i = 0; i < NDEC; ++i) mbar_init(bar(&sh.dec_read[i]), readers);
      for (int i = 0; i < NR; ++i)
        mbar_init(bar(&sh.ready[i]), QUANT ? nc + 1 : 2);  // the key tile, the S buffer
      for (int i = 0; i < NS; ++i) mbar_arrive(bar(&sh.ready[i]));  // S buffers free at first
      if constexpr (QUANT) {
        for (int i = 0; i < NV; ++i) mbar_init(bar(&sh.v_full[i]), nc);
        for (int i = 0; i < 3; ++i) {
          mbar_init(bar(&sh.kc_empty[i]), nc);
          mbar_init(bar(&sh.vc_empty[i]), nc);
        }
      }
      for (int i = 0; i < NS; ++i) mbar_init(bar(&sh.p_full[i]), nq);
      mbar_init(bar(&sh.l_full), nq);
      fence_mbar_init();
    }
  }
  if (warp == WARP_PV && lane == 0) {
    prefetch_tmap(&tm_q);
    if constexpr (!QUANT) {
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
    mbar_init(bar(&sh.q_full), 1);
    mbar_init(bar(&sh.q_ready), 8);
    mbar_init(bar(&sh.v_tail), 1);
    for (int i = 0; i < NR; ++i) mbar_init(bar(&sh.qk_done[i]), 1);
    for (int i = 0; i < NV; ++i) {
      if (!QUANT) mbar_init(bar(&sh.v_full[i]), 1);
      mbar_init(bar(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < NS; ++i) mbar_init(bar(&sh.pv_done[i]), 1);
    for (int i = 0; i < NDEC; ++i) mbar_init(bar(&sh.dec_full[i]), 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(&sh.kc_full[i]), 1);
      mbar_init(bar(&sh.vc_full[i]), 1);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(&sh.tmem_base), TMEM_COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  const TileInfo x = sh.tile;
  const int nb = x.nb;
  const int rows = x.s >= 0 ? x.ntok * a.G : 0;
  const bool dense = x.ln_lam == -INFINITY;
  // Quarters that have rows; the deciders (exponential warps) of the others help
  // the key (value) converters, so a decode step has seven of each.
  const int nq = REP ? NQ : (rows + 31) / 32, nc = 8 - nq, quarter = warp & 3;
  const bool k_conv = QUANT && ((warp >= WARP_KC && warp < WARP_VC) || (warp < NQ && quarter >= nq));
  const bool v_conv = QUANT && (warp >= WARP_VC || (warp >= NQ && warp < 2 * NQ && quarter >= nq));
  const int cw = warp >= WARP_KC ? quarter : 4 + quarter - nq;  // a converter's number
  // End of the query rows in [r, r + 16).
  auto q_end = [&](int r) { return min(r + 16, REP ? (r & ~31) + rows : rows); };

  if (blockIdx.x == 0 && (x.s < 0 || nb == 0) && warp == WARP_PV) check_batch(a, lane);
  if (x.s < 0) {
    // no tile for this CTA
  } else if (nb == 0) {
    // No visible key: O = 0, LSE = -inf (one split), or a partial of no weight.
#pragma unroll 1
    for (int i = tid; i < rows * (D / 8); i += C::WARPS * 32) {
      const int r = i / (D / 8);
      const int64_t orow = (int64_t)(x.tok0 + r / a.G) * a.Hq + hk * a.G + r % a.G;
      if (a.n_splits == 1)
        reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + orow * D)[i % (D / 8)] =
            make_uint4(0, 0, 0, 0);
      if (i % (D / 8) == 0)
        (a.n_splits == 1 ? a.lse : a.lse_part)[orow * a.n_splits + sp] = -INFINITY;
    }
  } else if (warp == WARP_K) {
    // ---------------------------------------------- query and key producer --
    fence_proxy_async_smem();  // the initialised barriers, for every lane's copies
    if (lane == 0) {
      const uint64_t once = policy_evict_first();
      constexpr int COPIES = REP ? 4 : 1;
      mbar_expect_tx(bar(&sh.q_full), COPIES * 2 * 128 * a.G * q_box_tokens);
      for (int i = 0; i < COPIES; ++i) {
        const uint32_t dst = base + L::Q + i * 32 * 128;
        tma_load_3d(dst, &tm_q, bar(&sh.q_full), 0, hk * a.G, x.tok0, once);
        tma_load_3d(dst + HALF_BYTES, &tm_q, bar(&sh.q_full), 64, hk * a.G, x.tok0, once);
      }
    }
    __syncwarp();
    int issued = 0;
#pragma unroll 1
    for (int c = 0; c < nb && !*abort; ++c) {
      // The ring's slot last held block c - K_AHEAD.
      if (c >= K_AHEAD &&
          !(QUANT ? wait_warp(&sh.kc_empty[c % NC], c / NC - 1)
                  : wait_warp(&sh.qk_done[(c - K_AHEAD) % NR], (c - K_AHEAD) / NR)))
        break;
      load_k(c);
      ++issued;
    }
    if (__any_sync(0xffffffffu, pages.bad) && lane == 0) atomicOr(a.err, kErrBadArg);
    if (lane == 0) {
      // Drain: the last load of each slot has landed before exit.
      mbar_wait_drain(bar(&sh.q_full), 0);
#pragma unroll 1
      for (int c = max(0, issued - K_AHEAD); c < issued; ++c)
        mbar_wait_drain(bar(k_bar(c)), (c / (QUANT ? NC : NR)) & 1);
    }
  } else if (warp == WARP_V) {
    // ------------------------------------------------------ value producer --
    fence_proxy_async_smem();
    int vi = 0;
    bool tail = false;
#pragma unroll 1
    for (int c = 0; c < nb && !*abort; ++c) {
      // A dense tile keeps every block: its values need no decision and load
      // as far ahead as their ring allows.
      if (!dense) {
        if (!wait_warp(&sh.dec_full[c % NDEC], c / NDEC)) break;
        const int keep = sh.dec[c % NDEC];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.dec_read[c % NDEC]));
        if (!keep) continue;
      }
      const int j = x.j0 + c;
      constexpr int N = QUANT ? NC : NV;
      const int s = vi % N;
      if (vi >= N && !wait_warp(QUANT ? &sh.vc_empty[s] : &sh.v_empty[s], vi / N - 1)) break;
      const uint32_t dst = base + (QUANT ? L::VC + s * L::VSTAGE : L::V + s * TILE_BYTES);
      const int left = x.kv - j * BN;  // rows of the block below kv
      // The last block, where its product does not end at kv: zero the rows behind.
      const bool cut = !QUANT && left < BN && (left & 15);
      load_block<FMT>(a, pages, &tm_v, true, j, dst,
                      bar(QUANT ? &sh.vc_full[s] : cut ? &sh.v_tail : &sh.v_full[s]), lane);
      if (cut) {
        tail = true;
        if (!wait_warp(&sh.v_tail, 0)) break;
#pragma unroll 1
        for (int i = lane; i < (-left & 15) * 16; i += 32)
          st_shared_v4(dst + (i & 8 ? HALF_BYTES : 0) + (left + (i >> 4)) * 128 + (i & 7) * 16, 0, 0,
                       0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.v_full[s]));
      }
      ++vi;
    }
    if (lane == 0) {
      constexpr int N = QUANT ? NC : NV;
      if (tail) mbar_wait_drain(bar(&sh.v_tail), 0);
#pragma unroll 1
      for (int s = 0; s < N && s < vi; ++s) {
        const int last = s + ((vi - 1 - s) / N) * N;
        mbar_wait_drain(bar(QUANT ? &sh.vc_full[s] : &sh.v_full[s]), (last / N) & 1);
      }
    }
  } else if (warp == WARP_MMA || (!QUANT && warp == WARP_MMA2)) {
    // ------------------------------------------------------ Q.K^T issuers --
    const int mine = warp == WARP_MMA ? 0 : 1;
    const bool ok = wait_warp(QUANT ? &sh.q_ready : &sh.q_full, 0);
    fence_after_sync();
    const uint64_t qdesc = kmajor_base(base + L::Q);
#pragma unroll 1
    for (int c = mine; ok && c < nb; c += QUANT ? 1 : 2) {
      if (!wait_warp(&sh.ready[c % NR], c / NR)) break;
      fence_after_sync();
      if (lane == 0) {
        const uint64_t kd = kmajor_base(base + L::K + (c % NKD) * TILE_BYTES);
        const uint32_t d_s = tmem + (c % NS) * BN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(d_s, qdesc + kmajor_step(kk), kd + kmajor_step(kk), QUANT ? IDESC_QK16 : IDESC_QK,
                      kk > 0);
        mma_commit(bar(&sh.qk_done[c % NR]));
      }
      __syncwarp();
    }
  } else if (warp == WARP_PV) {
    // ---------------------------------------------------------- P.V issuer --
    if (blockIdx.x == 0) check_batch(a, lane);
    if (lane == 0) {
      int kc = 0;
#pragma unroll 1
      for (int c = 0; c < nb && !*abort; ++c) {
        if (!wait(&sh.dec_full[c % NDEC], c / NDEC)) break;
        const int keep = sh.dec[c % NDEC];
        mbar_arrive(bar(&sh.dec_read[c % NDEC]));
        if (!keep) continue;
        const int pb = kc % NS, vs = kc % NV;
        if (!wait(&sh.p_full[pb], kc / NS) || !wait(&sh.v_full[vs], kc / NV)) break;
        fence_after_sync();
        const uint32_t pt = tmem + (c % NS) * BN;
        const uint64_t vd = vmajor_base(base + L::V + vs * TILE_BYTES);
        issue_pv(tmem + TMEM_O, pt, vd, QUANT ? IDESC_PV16 : IDESC_PV, kc > 0,
                 QUANT || c != nb - 1 ? BN : x.kv - (x.j0 + c) * BN);
        mma_commit(bar(&sh.v_empty[vs]));
        mma_commit(bar(&sh.ready[(c + NS) % NR]));  // S buffer free for block c + NS
        mma_commit(bar(&sh.pv_done[pb]));
        ++kc;
      }
    }
  } else if (k_conv) {
    // ------------------------------------------------------ key converters --
    if constexpr (QUANT) {
      if (cw < 4 && wait_warp(&sh.q_full, 0)) {
        convert_q(base + L::Q, cw * 16, q_end(cw * 16), lane, sh.qexp);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.q_ready));
      }
#pragma unroll 1
      for (int c = 0; c < nb; ++c) {
        if (!wait_warp(&sh.kc_full[c % NC], c / NC)) break;
        // The tile last fed block c - NKD's Q.K^T.
        if (c >= NKD && !wait_warp(&sh.qk_done[(c - NKD) % NR], (c - NKD) / NR)) break;
        const uint8_t *stage = smem_raw + L::KC + (c % NC) * L::KSTAGE;
        const int ek = block_top<FMT>(a, x, hk, x.j0 + c, false, stage + L::SCALES, lane);
        if (cw == 0) {
          const int ev = block_top<FMT>(a, x, hk, x.j0 + c, true, stage + L::SCALES + BN, lane);
          if (lane == 0) sh.esc[c % NE] = (uint16_t)(ek | (ev << 8));
        }
        convert_block<FMT>(stage, base + L::K + (c % NKD) * TILE_BYTES, cw, nc, lane, ek, BN);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(&sh.ready[c % NR]));
          mbar_arrive(bar(&sh.kc_empty[c % NC]));
        }
      }
    }
  } else if (v_conv) {
    // ---------------------------------------------------- value converters --
    if constexpr (QUANT) {
      if (cw < 4 && wait_warp(&sh.q_full, 0)) {
        convert_q(base + L::Q, 64 + cw * 16, q_end(64 + cw * 16), lane, sh.qexp);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.q_ready));
      }
      int vi = 0;
#pragma unroll 1
      for (int c = 0; c < nb && !*abort; ++c) {
        if (!dense) {
          if (!wait_warp(&sh.dec_full[c % NDEC], c / NDEC)) break;
          const int keep = sh.dec[c % NDEC];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh.dec_read[c % NDEC]));
          if (!keep) continue;
        }
        if (!wait_warp(&sh.vc_full[vi % NC], vi / NC)) break;
        if (vi >= NV && !wait_warp(&sh.v_empty[vi % NV], vi / NV - 1)) break;
        const uint8_t *stage = smem_raw + L::VC + (vi % NC) * L::VSTAGE;
        const int ev = block_top<FMT>(a, x, hk, x.j0 + c, true, stage + L::SCALES, lane);
        convert_block<FMT>(stage, base + L::V + (vi % NV) * TILE_BYTES, cw, nc, lane, ev,
                           x.kv - (x.j0 + c) * BN);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(&sh.v_full[vi % NV]));
          mbar_arrive(bar(&sh.vc_empty[vi % NC]));
        }
        ++vi;
      }
    }
  } else if (quarter < nq) {
    // ------------------------------------------------- deciders / exponentials --
    const bool decider = warp < NQ;
    const int r = quarter * 32 + lane;  // TMEM lane
    const int row = REP ? lane : r;     // row of the tile
    const bool valid = row < rows;
    const int tok = row / a.G;
    const int limit = a.causal && valid ? x.pos0 + tok + 1 : x.kv;  // the row sees keys below it
    const int min_limit = a.causal ? x.pos0 + 1 : x.kv;             // the tile's smallest
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const float sl2 = a.scale * kLog2e;
    // Running maxima: of the row maxima, of (row max + E_v) (the same over bf16 rows);
    // the exponentials' references, which lag behind them; row sum.
    float t2 = -INFINITY, y2 = -INFINITY;
    float mref = -INFINITY, yref = -INFINITY, l = 0.f;
    int kc = 0;
    bool ok = true;
    // A quantised cache: raw score to log2 units for a block of key exponent E_k,
    // sl2 * 2^(E_k - x) (kept normal, so that a masked score stays -inf).
    int qx = 0;
    if constexpr (QUANT) {
      ok = wait_warp(&sh.q_ready, 0);
      qx = sh.qexp[r] + 127;
    }
    auto block_sl2 = [&](int ek) {
      const int e = max(-126, min(126, ek - qx));
      return fmaxf(sl2 * __int_as_float((e + 127) << 23), 1.17549435e-38f);
    };

    if (decider) {
      const float c2 = x.ln_lam * kLog2e;
      float m2 = -INFINITY;  // running max (log2 units)
      uint32_t word = 0;
      uint32_t *bits = a.bits ? a.bits + ((((int64_t)x.s * a.Hkv + hk) * a.n_t + x.t) * a.n_splits + sp) * a.words
                              : nullptr;
#pragma unroll 1
      for (int c = 0; c < nb; ++c) {
        // After a failed wait the loop still runs to its end, so that the
        // warps meet the vote barrier equally often.
        if (ok) ok = wait_warp(&sh.qk_done[c % NR], c / NR);
        bool keep_vote = false;
        if (ok) {
          fence_after_sync();
          const uint32_t sa = lane_base + (c % NS) * BN + (REP ? 32 * quarter : 0);
          const int key0 = (x.j0 + c) * BN + (REP ? 32 * quarter : 0);
          if (key0 + (REP ? 32 : BN) > min_limit) mask_block_tmem(sa, limit - key0, REP ? 1 : 4);
          float mt;
          if constexpr (REP) {
            uint32_t x0[32];
            tmem_ld32(sa, x0);
            tmem_wait_ld_regs(x0);
            mt = chunk_max(x0);
          } else if constexpr (QUANT) {  // 20 warps: fewer registers a thread
            mt = -INFINITY;
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t x0[32], x1[32];
              tmem_ld32(sa + 64 * hh, x0);
              tmem_ld32(sa + 64 * hh + 32, x1);
              tmem_wait_ld_regs(x0);
              tmem_wait_ld_regs(x1);
              mt = max3_nan(mt, chunk_max(x0), chunk_max(x1));
            }
          } else {
            uint32_t x0[32], x1[32], x2[32], x3[32];
            tmem_ld32(sa, x0);
            tmem_ld32(sa + 32, x1);
            tmem_ld32(sa + 64, x2);
            tmem_ld32(sa + 96, x3);
            tmem_wait_ld_regs(x0);
            tmem_wait_ld_regs(x1);
            tmem_wait_ld_regs(x2);
            tmem_wait_ld_regs(x3);
            mt = max_nan(max_nan(chunk_max(x0), chunk_max(x1)), max_nan(chunk_max(x2), chunk_max(x3)));
          }
          const float bl2 = QUANT ? block_sl2(sh.esc[c % NE] & 255) : sl2;
          if constexpr (REP) {
            if (!dense) {  // the rows' maxima over all four quarters' keys
              sh.mdec[2][r] = mt;  // (read before the vote barrier of the last block)
              named_bar_sync(kDeciderBarrier, NQ * 32);
              mt = max_nan(max_nan(sh.mdec[2][lane], sh.mdec[2][32 + lane]),
                           max_nan(sh.mdec[2][64 + lane], sh.mdec[2][96 + lane]));
            }
          } else {
            t2 = fmaxf(t2, mt * bl2);
            sh.mdec[c % NS][r] = QUANT ? mt * bl2 : t2;
          }
          const float pm2 = mt * bl2;
          // With ln(lambda) < 0, "rowmax - m_new < c" is "rowmax - m_old < c".
          const float diff = mt == -INFINITY ? -INFINITY : pm2 - m2;
          keep_vote = dense || !__all_sync(0xffffffffu, !valid || diff < c2 || mt == -INFINITY);
          m2 = max_nan(m2, pm2);
          fence_before_sync();  // this warp's reads of S_j are complete
        } else if (REP && !dense) {
          named_bar_sync(kDeciderBarrier, NQ * 32);
        }
        const bool keep = bar_red_or(kDeciderBarrier, nq * 32, keep_vote);
        if (!ok) continue;
        if (lane == 0 && warp == (nq == NQ ? c & (NQ - 1) : 0)) {
          if (!keep) mbar_arrive(bar(&sh.ready[(c + NS) % NR]));  // its S buffer is free
          if (c < NDEC || wait(&sh.dec_read[c % NDEC], c / NDEC - 1)) {
            sh.dec[c % NDEC] = keep ? 1 : 0;
            mbar_arrive(bar(&sh.dec_full[c % NDEC]));
          }
        }
        if (tid == 0 && bits) {
          if (!keep) word |= 1u << (c & 31);
          if ((c & 31) == 31 || c == nb - 1) {
            bits[c >> 5] = word;
            word = 0;
          }
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < nb; ++c) {
        if (!wait_warp(&sh.dec_full[c % NDEC], c / NDEC)) {
          ok = false;
          break;
        }
        const int keep = sh.dec[c % NDEC];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.dec_read[c % NDEC]));
        if (!keep) continue;
        fence_after_sync();
        const uint32_t sa = lane_base + (c % NS) * BN;  // masked by the deciders
        float e_v = 0.f, bl2 = sl2;
        if constexpr (QUANT) {
          const int e = sh.esc[c % NE];
          e_v = e >> 8 ? (float)((e >> 8) - 127) : -INFINITY;
          bl2 = block_sl2(e & 255);
        }
        uint32_t own[REP ? 32 : 1];  // REP: the scores of the quarter's 32 keys
        float mrow;
        if constexpr (REP) {
          tmem_ld32(sa + 32 * quarter, own);
          tmem_wait_ld_regs(own);
          mrow = chunk_max(own) * bl2;
        } else {
          mrow = sh.mdec[c % NS][r];
        }
        t2 = fmaxf(t2, mrow);
        bool rescale = false;
        float alpha = 1.f, lalpha = 1.f;  // of O, of l
        auto follow = [&](float &ref, float now, float &factor) {
          if (ref == -INFINITY) {
            ref = now;
          } else if (valid && now > ref + kRescaleLog2) {
            factor = ex2(ref - now);
            ref = now;
            return true;
          }
          return false;
        };
        float f = 0.f;  // P is 2^f times a weight
        if constexpr (QUANT) {
          y2 = fmaxf(y2, mrow + e_v);
          follow(mref, t2, lalpha);
          rescale = follow(yref, y2, alpha);
          // (Below 2^-40 P is 0 in fp16, whatever the weight, which has to stay in fp32's
          // range; above 2^100 the weights are below 2^-85, and what is lost of them is
          // nothing beside the row sum.)
          if (yref != -INFINITY) f = fmaxf(mref + e_v - yref + kPLog2, -40.f);
        } else {
          rescale = follow(mref, t2, alpha);
          lalpha = alpha;
        }
        // A row without a visible key so far has only -inf scores: P = 0.
        const float nref = mref == -INFINITY ? 0.f : f - mref;
        const uint64_t sl2x2 = f2(bl2, bl2), negref2 = f2(nref, nref);
        uint64_t acc2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        if constexpr (REP) {
          // The quarter's 32 keys; zeros for the others (their scores in these
          // lanes have no reader).
          uint32_t pk[16], zero[16];
          chunk_exp<QUANT>(own, sl2x2, negref2, acc2, pk);
#pragma unroll
          for (int i = 0; i < 16; ++i) zero[i] = 0u;
          tmem_st16(sa + 16 * quarter, pk);
#pragma unroll
          for (int i = 1; i < 4; ++i) tmem_st16(sa + 16 * ((quarter + i) & 3), zero);
        } else if constexpr (QUANT) {
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t s[32], pk[32];
            tmem_ld32(sa + 64 * hh, s);
            tmem_wait_ld_regs(s);
            chunk_exp<true>(s, sl2x2, negref2, acc2, pk);
            tmem_ld32(sa + 64 * hh + 32, s);
            tmem_wait_ld_regs(s);
            chunk_exp<true>(s, sl2x2, negref2, acc2, pk + 16);
            tmem_st32(sa + 32 * hh, pk);
          }
        } else {
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            // The P pairs of keys [64 hh, 64 hh + 64) land in columns [32 hh,
            // 32 hh + 32), whose scores this or the previous half has loaded.
            uint32_t s0[32], s1[32], pk[32];
            tmem_ld32(sa + 64 * hh, s0);
            tmem_ld32(sa + 64 * hh + 32, s1);
            tmem_wait_ld_regs(s0);
            tmem_wait_ld_regs(s1);
            chunk_exp<false>(s0, sl2x2, negref2, acc2, pk);
            chunk_exp<false>(s1, sl2x2, negref2, acc2, pk + 16);
            tmem_st32(sa + 32 * hh, pk);
          }
        }
        tmem_wait_st();
        float acc[4];
        f2_split(acc2[0], acc[0], acc[1]);
        f2_split(acc2[1], acc[2], acc[3]);
        float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if constexpr (QUANT) sum *= ex2(-f);
        l = l * lalpha + sum;
        if (__any_sync(0xffffffffu, rescale) && kc >= 1) {
          if (!wait_warp(&sh.pv_done[(kc - 1) % NS], (kc - 1) / NS)) {
            ok = false;
            break;
          }
          fence_after_sync();
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            const uint32_t oa = lane_base + TMEM_O + cc * 32;
            tmem_ld32(oa, o);
            tmem_wait_ld_regs(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(oa, o);
          }
          tmem_wait_st();
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.p_full[kc % NS]));
        ++kc;
      }
      if (ok && kc > 0) ok = wait_warp(&sh.pv_done[(kc - 1) % NS], (kc - 1) / NS);
      // No kept block: O was never written.
      sh.mdec[0][r] = kc > 0 ? l : 0.f;
      sh.mdec[1][r] = mref;
      if constexpr (QUANT) sh.mdec[2][r] = yref;
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh.l_full));
    }

    // ---- epilogue: deciders take O columns [0,64), exponential warps [64,128)
    if (ok) ok = wait_warp(&sh.l_full, 0);
    const int64_t orow = (int64_t)(x.tok0 + tok) * a.Hq + hk * a.G + (row - tok * a.G);
    const int col0 = decider ? 0 : 64;
    // Four consecutive columns of an output row.
    auto put = [&](int64_t at, int col, float v0, float v1, float v2, float v3) {
      if (a.n_splits == 1)
        *reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.o + at * D + col) =
            make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
      else
        *reinterpret_cast<float4 *>(a.o_part + (at * a.n_splits + sp) * D + col) =
            make_float4(v0, v1, v2, v3);
    };
    float lrow = 0.f, lref = -INFINITY, w = 0.f;  // row sum, its reference, this lane's weight
    if (ok) {
      fence_after_sync();
      if constexpr (REP) {  // merge the quarters' states
        float lq[NQ], mq[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          lq[i] = sh.mdec[0][i * 32 + lane];
          mq[i] = sh.mdec[1][i * 32 + lane];
          // A quarter that met no key of the row has no say in the reference.
          if (lq[i] != 0.f) lref = fmaxf(lref, mq[i]);
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const float wi = lq[i] == 0.f ? 0.f : ex2(mq[i] - lref);
          lrow += lq[i] * wi;
          if (i == quarter) w = wi;
        }
      } else {
        lrow = sh.mdec[0][r];
        lref = sh.mdec[1][r];
        w = lrow == 0.f ? 0.f : 1.f;  // no key kept for this row: O = 0
      }
      if (QUANT && w != 0.f) w = ex2(sh.mdec[2][r] - lref - kPLog2);
      const float inv = lrow == 0.f ? 0.f : w / lrow;
      const bool none = w == 0.f;  // (the accumulator may hold anything)
      // The rows leave through 4 KB of the query tile a warp (free by now): a lane's
      // row in 16-byte pieces, then 128-byte runs of four rows an instruction.
      const uint32_t stage = base + L::Q + warp * 4096;
      auto put_row = [&](int piece, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
        st_shared_v4(stage + lane * 128 + ((piece ^ (lane & 7)) * 16), v0, v1, v2, v3);
      };
      auto store_rows = [&](uint8_t *out, int64_t row_bytes) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int l2 = it * 4 + (lane >> 3), piece = lane & 7;
          const int64_t at = __shfl_sync(0xffffffffu, orow, l2);
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(stage + l2 * 128 + ((piece ^ (l2 & 7)) * 16))
                       : "memory");
          if (quarter * 32 + l2 < rows) *reinterpret_cast<uint4 *>(out + at * row_bytes + piece * 16) = v;
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t o[32];
        const int col = col0 + cc * 32;
        tmem_ld32(lane_base + TMEM_O + col, o);
        tmem_wait_ld_regs(o);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          o[i] = none ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
        if constexpr (REP) {
          if (!valid) continue;
          const uint32_t at = base + (uint32_t)((r * MERGE_STRIDE + col) * 4);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared_v4(at + q * 16, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        } else if (a.n_splits == 1) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            put_row(cc * 4 + q, pack_bf16x2(__uint_as_float(o[8 * q]), __uint_as_float(o[8 * q + 1])),
                    pack_bf16x2(__uint_as_float(o[8 * q + 2]), __uint_as_float(o[8 * q + 3])),
                    pack_bf16x2(__uint_as_float(o[8 * q + 4]), __uint_as_float(o[8 * q + 5])),
                    pack_bf16x2(__uint_as_float(o[8 * q + 6]), __uint_as_float(o[8 * q + 7])));
          if (cc == 1) store_rows((uint8_t *)a.o + col0 * 2, D * 2);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            put_row(q, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          store_rows((uint8_t *)(a.o_part + (int64_t)sp * D + col), (int64_t)a.n_splits * D * 4);
        }
      }
      if (valid && !decider && (!REP || quarter == 0))
        (a.n_splits == 1 ? a.lse : a.lse_part)[orow * a.n_splits + sp] =
            lrow == 0.f ? -INFINITY : lref * kLn2 + logf(lrow);
    }
    if constexpr (REP) {
      // The four quarters' weighted rows stand in the query, key and value tiles,
      // which nothing reads any more; 256 threads add them up, four columns each.
      named_bar_sync(kMergeBarrier, 2 * NQ * 32);
      if (ok) {
#pragma unroll 1
        for (int i = tid; i < rows * (D / 4); i += 2 * NQ * 32) {
          const int rr = i / (D / 4), col = i % (D / 4) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const float4 u = *reinterpret_cast<const float4 *>(
                smem_raw + ((q * 32 + rr) * MERGE_STRIDE + col) * 4);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          const int t = rr / a.G;
          put((int64_t)(x.tok0 + t) * a.Hq + hk * a.G + (rr - t * a.G), col, v.x, v.y, v.z, v.w);
        }
      }
    }
  }

  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == WARP_MMA) {
    fence_after_sync();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------ bf16 prompts --
// Tiles of more than 32 rows over a bf16 cache (prompts, chunks of them, and the
// widened rows of a quantised cache): the same loop, in CTAs that stay.  A CTA that
// has issued its tile's key loads takes over a CTA of the grid that has not started
// (cluster launch control) and goes on to load that one's queries and keys, so that
// set-up, the first loads and the first scores of a tile lie under the end of the
// one before, and TMEM and barriers are set up once.  Rings run on from tile to
// tile: block g is the CTA's g-th.  Two query tiles (an epilogue puts its rows in
// order where its queries were), three key and two value tiles.
// Bound for short tiles: the scores' way to the last P.V and out, which the next
// tile's decisions wait for.
constexpr int PK = 3, PQ = 2;
constexpr uint32_t P_Q = 0, P_K = PQ * TILE_BYTES, P_V = P_K + PK * TILE_BYTES;
constexpr uint32_t P_END = P_V + NV * TILE_BYTES;
constexpr int P_WARPS = 13;
constexpr int kTileBarrier = 2;
// In the place of a row's first LSE: its outputs are written (a NaN that no
// computation gives).
constexpr uint32_t kWholeRow = 0x7fc5a5a5u;

struct PromptShared {
  uint4 next;            // answer of the cluster launch control
  uint64_t next_full;
  uint64_t tile_full[2];   // ring of the tiles: set, ..
  uint64_t tile_empty[2];  // .. left by twelve warps (all but the key producer)
  uint64_t q_full[2];
  uint64_t ready[NR];    // slot g % NR: block g's key tile is in and its S buffer free
  uint64_t qk_done[NR];
  uint64_t v_full[NV], v_empty[NV];
  uint64_t p_full[NS], pv_done[NS];
  uint64_t dec_full[NDEC], dec_read[NDEC];
  uint64_t l_full[2];
  uint64_t v_tail;
  int dec[NDEC];
  float mdec[NS][BM];    // running max after the buffer's block (log2 units)
  float sum[BM], ref[BM];  // row sums and references for the epilogue
  TileInfo tile[2];
  int hk[2], sp[2];      // KV head; split, -1: the rows go to the outputs
  uint32_t word;         // the bitmap's current word
  uint32_t tmem_base;
  int abort;
};
static_assert(P_END + sizeof(PromptShared) <= 227 * 1024, "shared memory budget");

// Asks for a CTA of this grid that has not started; the answer lands in `at` and
// completes 16 bytes on `b`.
__device__ __forceinline__ void take_cta(uint32_t at, uint32_t b) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(at),
      "r"(b)
      : "memory");
}
// The taken CTA's blockIdx.x, or -1: none was left.
__device__ __forceinline__ int taken_cta(uint32_t at) {
  uint32_t some, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(some), "=r"(x)
      : "r"(at)
      : "memory");
  return some ? (int)x : -1;
}

// SPLIT: n_splits > 1.
template <bool SPLIT>
__global__ void __launch_bounds__(P_WARPS * 32, 1)
    prompt_paged_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ ChunkArgs a, const int q_box_tokens) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PromptShared &sh = *reinterpret_cast<PromptShared *>(smem_raw + P_END);
  const uint32_t base = smem_u32(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (base & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (tid == 0) atomicOr(a.err, kErrLayout);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits for this grid's end)
  volatile int *abort = &sh.abort;
  auto bar = [&](uint64_t *b) { return smem_u32(b); };
  auto wait = [&](uint64_t *b, unsigned phase) {
    return mbar_wait_shared(smem_u32(b), phase & 1, abort, a.err);
  };
  auto wait_warp = [&](uint64_t *b, unsigned phase) {
    return __all_sync(0xffffffffu, mbar_wait_shared(smem_u32(b), phase & 1, abort, a.err));
  };

  Producer pages;  // of the two producer warps
  TileInfo found{};  // the key producer's first tile
  int unit = (int)blockIdx.x;
  if (warp == WARP_K) {
    found = producer_tile(a, pages, unit / a.Hkv, 0, unit % a.Hkv, lane);
  } else if (warp == WARP_PV && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    mbar_init(bar(&sh.next_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh.tile_full[i]), 1);
      mbar_init(bar(&sh.tile_empty[i]), P_WARPS - 1);
      mbar_init(bar(&sh.q_full[i]), 1);
      mbar_init(bar(&sh.l_full[i]), NQ);
    }
    mbar_init(bar(&sh.v_tail), 1);
    for (int i = 0; i < NR; ++i) {
      mbar_init(bar(&sh.ready[i]), 2);  // the key tile, the S buffer
      mbar_init(bar(&sh.qk_done[i]), 1);
    }
    for (int i = 0; i < NS; ++i) mbar_arrive(bar(&sh.ready[i]));  // S buffers free at first
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar(&sh.v_full[i]), 1);
      mbar_init(bar(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(&sh.p_full[i]), NQ);
      mbar_init(bar(&sh.pv_done[i]), 1);
    }
    for (int i = 0; i < NDEC; ++i) {
      mbar_init(bar(&sh.dec_full[i]), 1);
      mbar_init(bar(&sh.dec_read[i]), 2 + NQ);  // both value warps, the exponential warps
    }
    sh.abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(&sh.tmem_base), TMEM_COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  if (blockIdx.x == 0 && warp == WARP_PV) check_batch(a, lane);

  if (warp == WARP_K) {
    // ------------------------------------------ tiles; queries and keys --
    fence_proxy_async_smem();
    const uint64_t once = policy_evict_first();
    unsigned it = 0, g = 0, asked = 0;
    auto ask = [&]() {
      if (lane == 0) {
        mbar_expect_tx(bar(&sh.next_full), 16);
        take_cta(smem_u32(&sh.next), bar(&sh.next_full));
      }
      __syncwarp();
      ++asked;
    };
#pragma unroll 1
    while (true) {
      const int hk = unit % a.Hkv;
      if (asked) found = producer_tile(a, pages, unit / a.Hkv, 0, hk, lane);
      // The tile's splits, one after the other; those without a block are a partial of
      // no weight (where there is one split: O = 0, LSE = -inf).  A dense tile needs no
      // cut: its rows go to the outputs, and the merge leaves them alone.
      const int blocks = (found.kv + BN - 1) / BN, rows = found.s >= 0 ? found.ntok * a.G : 0;
      const bool whole = found.ln_lam == -INFINITY;
      const int run = !SPLIT || whole ? blocks : a.bps;
      const int splits = !rows || !blocks ? 0 : SPLIT ? (blocks + run - 1) / run : 1;
      if (splits == 0) ask();
      bool ok = true;
#pragma unroll 1
      for (int sp = 0; sp < splits && ok; ++sp, ++it) {
        const unsigned slot = it & 1;
        found.j0 = sp * run;
        found.nb = min(blocks - found.j0, run);
        ok = it < 2 || wait_warp(&sh.tile_empty[slot], (it >> 1) - 1);
        if (!ok) break;
        if (lane == 0) {
          sh.tile[slot] = found;
          sh.hk[slot] = hk;
          sh.sp[slot] = SPLIT && !whole ? sp : -1;
          mbar_arrive(bar(&sh.tile_full[slot]));
          mbar_expect_tx(bar(&sh.q_full[slot]), 2 * 128 * a.G * q_box_tokens);
          const uint32_t dst = base + P_Q + slot * TILE_BYTES;
          tma_load_3d(dst, &tm_q, bar(&sh.q_full[slot]), 0, hk * a.G, found.tok0, once);
          tma_load_3d(dst + HALF_BYTES, &tm_q, bar(&sh.q_full[slot]), 64, hk * a.G, found.tok0, once);
        }
        __syncwarp();
        // The next CTA as late as may be, so that the last ones share what is left:
        // with the last keys that the ring can take.
        const int ask_at = sp == splits - 1 ? max(0, found.nb - PK) : -1;
#pragma unroll 1
        for (int c = 0; c < found.nb; ++c, ++g) {
          if (c == ask_at) ask();
          ok = g < PK || wait_warp(&sh.qk_done[(g - PK) % NR], (g - PK) / NR);
          if (!ok) break;
          load_block_here<kKvBf16>(a, pages, &tm_k, false, found.j0 + c,
                                   base + P_K + (g % PK) * TILE_BYTES, bar(&sh.ready[g % NR]), lane);
        }
      }
      if (__any_sync(0xffffffffu, pages.bad) && lane == 0) atomicOr(a.err, kErrBadArg);
      if (!ok) break;
      if (splits < (!SPLIT || whole ? 1 : a.n_splits)) {
#pragma unroll 1
        for (int r = lane; r < rows; r += 32) {
          const int tok = r / a.G;
          const int64_t orow = (int64_t)(found.tok0 + tok) * a.Hq + hk * a.G + (r - tok * a.G);
          if constexpr (!SPLIT) {
#pragma unroll 1
            for (int i = 0; i < D / 8; ++i)
              reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + orow * D)[i] = make_uint4(0, 0, 0, 0);
          }
          float *lse = SPLIT ? a.lse_part + orow * a.n_splits : a.lse + orow;
#pragma unroll 1
          for (int sp = splits; sp < (SPLIT ? a.n_splits : 1); ++sp) lse[sp] = -INFINITY;
        }
      }
      if (!wait_warp(&sh.next_full, asked - 1)) break;
      unit = taken_cta(smem_u32(&sh.next));
      __syncwarp();
      fence_proxy_async_smem();
      if (unit == 0) check_batch(a, lane);  // (that CTA's part)
      if (unit < 0) {
        const unsigned slot = it & 1;
        if (it >= 2 && !wait_warp(&sh.tile_empty[slot], (it >> 1) - 1)) break;
        if (lane == 0) {
          sh.tile[slot].s = -1;
          mbar_arrive(bar(&sh.tile_full[slot]));
        }
        break;
      }
    }
    if (lane == 0) {
      // Drain: the last answer and the last load of each slot have landed before exit.
      if (asked) mbar_wait_drain(bar(&sh.next_full), (asked - 1) & 1);
#pragma unroll 1
      for (unsigned i = it < 2 ? 0 : it - 2; i < it; ++i) mbar_wait_drain(bar(&sh.q_full[i & 1]), (i >> 1) & 1);
#pragma unroll 1
      for (unsigned i = g < PK ? 0 : g - PK; i < g; ++i) mbar_wait_drain(bar(&sh.ready[i % NR]), (i / NR) & 1);
    }
  } else if (warp == WARP_V) {
    // ------------------------------------------------------ value producer --
    fence_proxy_async_smem();
    unsigned vi = 0, g = 0, tails = 0;
    bool ok = true;
#pragma unroll 1
    for (unsigned it = 0; ok; ++it) {
      if (!wait_warp(&sh.tile_full[it & 1], it >> 1)) break;
      const TileInfo x = sh.tile[it & 1];
      if (x.s < 0) break;
      const bool dense = x.ln_lam == -INFINITY;
      producer_at(a, pages, x, sh.hk[it & 1], lane);
#pragma unroll 1
      for (int c = 0; c < x.nb; ++c, ++g) {
        // A dense tile keeps every block: its values need no decision.
        if (!dense) {
          ok = wait_warp(&sh.dec_full[g % NDEC], g / NDEC);
          if (!ok) break;
          const int keep = sh.dec[g % NDEC];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh.dec_read[g % NDEC]));
          if (!keep) continue;
        }
        const int j = x.j0 + c;
        const unsigned s = vi % NV;
        ok = vi < NV || wait_warp(&sh.v_empty[s], vi / NV - 1);
        if (!ok) break;
        const uint32_t dst = base + P_V + s * TILE_BYTES;
        const int left = x.kv - j * BN;  // rows of the block below kv
        // The last block, where its product does not end at kv: zero the rows behind.
        const bool cut = left < BN && (left & 15);
        load_block_here<kKvBf16>(a, pages, &tm_v, true, j, dst,
                                 bar(cut ? &sh.v_tail : &sh.v_full[s]), lane);
        if (cut) {
          ok = wait_warp(&sh.v_tail, tails++);
          if (!ok) break;
#pragma unroll 1
          for (int i = lane; i < (-left & 15) * 16; i += 32)
            st_shared_v4(dst + (i & 8 ? HALF_BYTES : 0) + (left + (i >> 4)) * 128 + (i & 7) * 16, 0, 0,
                         0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh.v_full[s]));
        }
        ++vi;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh.tile_empty[it & 1]));
    }
    if (lane == 0) {
      if (tails) mbar_wait_drain(bar(&sh.v_tail), (tails - 1) & 1);
#pragma unroll 1
      for (unsigned i = vi < NV ? 0 : vi - NV; i < vi; ++i) mbar_wait_drain(bar(&sh.v_full[i % NV]), (i / NV) & 1);
    }
  } else if (warp == WARP_MMA || warp == WARP_MMA2) {
    // ------------------------------------------------------ Q.K^T issuers --
    const unsigned mine = warp == WARP_MMA ? 0 : 1;
    unsigned g0 = 0;
    bool ok = true;
#pragma unroll 1
    for (unsigned it = 0; ok; ++it) {
      if (!wait_warp(&sh.tile_full[it & 1], it >> 1)) break;
      const int s = sh.tile[it & 1].s, nb = sh.tile[it & 1].nb;
      if (s < 0 || !wait_warp(&sh.q_full[it & 1], it >> 1)) break;
      fence_after_sync();
      const uint64_t qdesc = kmajor_base(base + P_Q + (it & 1) * TILE_BYTES);
#pragma unroll 1
      for (unsigned g = g0 + ((g0 ^ mine) & 1); g < g0 + nb; g += 2) {
        ok = wait_warp(&sh.ready[g % NR], g / NR);
        if (!ok) break;
        fence_after_sync();
        if (lane == 0) {
          const uint64_t kd = kmajor_base(base + P_K + (g % PK) * TILE_BYTES);
          const uint32_t d_s = tmem + (g % NS) * BN;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(d_s, qdesc + kmajor_step(kk), kd + kmajor_step(kk), IDESC_QK, kk > 0);
          mma_commit(bar(&sh.qk_done[g % NR]));
        }
        __syncwarp();
      }
      g0 += nb;
      if (lane == 0) mbar_arrive(bar(&sh.tile_empty[it & 1]));
    }
  } else if (warp == WARP_PV) {
    // ---------------------------------------------------------- P.V issuer --
    if (lane == 0) {
      unsigned kc = 0, g = 0;
      bool ok = true;
#pragma unroll 1
      for (unsigned it = 0; ok; ++it) {
        if (!wait(&sh.tile_full[it & 1], it >> 1)) break;
        const int s = sh.tile[it & 1].s, nb = sh.tile[it & 1].nb;
        if (s < 0) break;
        const int keys = sh.tile[it & 1].kv - sh.tile[it & 1].j0 * BN;
        bool first = true;
#pragma unroll 1
        for (int c = 0; c < nb; ++c, ++g) {
          ok = wait(&sh.dec_full[g % NDEC], g / NDEC);
          if (!ok) break;
          const int keep = sh.dec[g % NDEC];
          mbar_arrive(bar(&sh.dec_read[g % NDEC]));
          if (!keep) continue;
          const unsigned pb = kc % NS, vs = kc % NV;
          // O is the last tile's until its epilogue has read it.
          if (first && it) ok = wait(&sh.tile_empty[(it - 1) & 1], (it - 1) >> 1);
          ok = ok && wait(&sh.p_full[pb], kc / NS) && wait(&sh.v_full[vs], kc / NV);
          if (!ok) break;
          fence_after_sync();
          const uint32_t pt = tmem + (g % NS) * BN;
          const uint64_t vd = vmajor_base(base + P_V + vs * TILE_BYTES);
          issue_pv(tmem + TMEM_O, pt, vd, IDESC_PV, !first, c != nb - 1 ? BN : keys - c * BN);
          mma_commit(bar(&sh.v_empty[vs]));
          mma_commit(bar(&sh.ready[(g + NS) % NR]));  // S buffer free for block g + NS
          mma_commit(bar(&sh.pv_done[pb]));
          ++kc;
          first = false;
        }
        mbar_arrive(bar(&sh.tile_empty[it & 1]));
      }
    }
  } else {
    // ------------------------------------------------- deciders / exponentials --
    const bool decider = warp < NQ;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // TMEM lane, row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const float sl2 = a.scale * kLog2e;
    unsigned g = 0, kc = 0;  // blocks; of those, kept
    bool ok = true;
#pragma unroll 1
    for (unsigned it = 0;; ++it) {
      ok = ok && wait_warp(&sh.tile_full[it & 1], it >> 1);
      if (decider ? bar_red_or(kTileBarrier, NQ * 32, !ok) : !ok) break;  // (deciders meet at votes)
      // Read again where it is used: the loops need the registers.
      const TileInfo &x = sh.tile[it & 1];
      if (x.s < 0) break;
      const int nb = x.nb;
      const int nq = (x.ntok * a.G + 31) / 32;  // quarters that have rows
      const bool valid = r < x.ntok * a.G;
      if (quarter >= nq) {
        // A quarter without rows has no decider; its exponential warp follows the
        // decisions, to keep count.
        if (decider) {
          g += nb;
        } else {
#pragma unroll 1
          for (int c = 0; c < nb && ok; ++c, ++g) {
            ok = wait_warp(&sh.dec_full[g % NDEC], g / NDEC);
            const int keep = sh.dec[g % NDEC];
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(&sh.dec_read[g % NDEC]));
              if (keep) mbar_arrive(bar(&sh.p_full[kc % NS]));
            }
            if (keep) ++kc;
          }
          if (lane == 0) mbar_arrive(bar(&sh.l_full[it & 1]));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.tile_empty[it & 1]));
        continue;
      }
      if (decider) {
        const bool dense = x.ln_lam == -INFINITY;
        const int tok = r / a.G;
        const int key0 = x.j0 * BN;
        // The row sees keys below key0 + limit; the tile's smallest limit.
        const int limit = (a.causal && valid ? x.pos0 + tok + 1 : x.kv) - key0;
        const int min_limit = (a.causal ? x.pos0 + 1 : x.kv) - key0;
        const float c2 = x.ln_lam * kLog2e;
        float m2 = -INFINITY;  // running max (log2 units)
#pragma unroll 1
        for (int c = 0; c < nb; ++c, ++g) {
          // After a failed wait the loop still runs to its end, so that the
          // warps meet the vote barrier equally often.
          if (ok) ok = wait_warp(&sh.qk_done[g % NR], g / NR);
          bool keep_vote = false;
          if (ok) {
            fence_after_sync();
            const uint32_t sa = lane_base + (g % NS) * BN;
            if (c * BN + BN > min_limit) mask_block_tmem(sa, limit - c * BN, 4);
            float mt = -INFINITY;
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t x0[32], x1[32];
              tmem_ld32(sa + 64 * hh, x0);
              tmem_ld32(sa + 64 * hh + 32, x1);
              tmem_wait_ld_regs(x0);
              tmem_wait_ld_regs(x1);
              mt = max3_nan(mt, chunk_max(x0), chunk_max(x1));
            }
            const float pm2 = mt * sl2;
            // With ln(lambda) < 0, "rowmax - m_new < c" is "rowmax - m_old < c".
            const float diff = mt == -INFINITY ? -INFINITY : pm2 - m2;
            keep_vote = dense || !__all_sync(0xffffffffu, !valid || diff < c2 || mt == -INFINITY);
            m2 = max_nan(m2, pm2);
            sh.mdec[g % NS][r] = m2;
            fence_before_sync();  // this warp's reads of S are complete
          }
          const bool keep = bar_red_or(kDeciderBarrier, nq * 32, keep_vote);
          if (!ok) continue;
          if (lane == 0 && warp == (nq == NQ ? c & (NQ - 1) : 0)) {
            if (!keep) mbar_arrive(bar(&sh.ready[(g + NS) % NR]));  // its S buffer is free
            if (g < NDEC || wait(&sh.dec_read[g % NDEC], g / NDEC - 1)) {
              sh.dec[g % NDEC] = keep ? 1 : 0;
              mbar_arrive(bar(&sh.dec_full[g % NDEC]));
              if (dense) mbar_arrive(bar(&sh.dec_read[g % NDEC]));  // the value producer does not read it
            }
          }
          if (tid == 0 && a.bits && !dense) {
            const uint32_t word = ((c & 31) ? sh.word : 0u) | (keep ? 0u : 1u << (c & 31));
            sh.word = word;
            if ((c & 31) == 31 || c == nb - 1) {
              const int64_t tile = ((int64_t)x.s * a.Hkv + sh.hk[it & 1]) * a.n_t + x.t;
              a.bits[(tile * a.n_splits + (SPLIT ? sh.sp[it & 1] : 0)) * a.words + (c >> 5)] = word;
            }
          }
        }
      } else {
        float mref = -INFINITY, l = 0.f;
        const unsigned kc0 = kc;
#pragma unroll 1
        for (int c = 0; c < nb; ++c, ++g) {
          ok = wait_warp(&sh.dec_full[g % NDEC], g / NDEC);
          if (!ok) break;
          const int keep = sh.dec[g % NDEC];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh.dec_read[g % NDEC]));
          if (!keep) continue;
          fence_after_sync();
          const uint32_t sa = lane_base + (g % NS) * BN;  // masked by the deciders
          const float mnew = sh.mdec[g % NS][r];
          bool rescale = false;
          float alpha = 1.f;
          if (mref == -INFINITY) {
            mref = mnew;
          } else if (valid && mnew > mref + kRescaleLog2) {
            alpha = ex2(mref - mnew);
            mref = mnew;
            rescale = true;
          }
          // A row without a visible key so far has only -inf scores: P = 0.
          const float nref = mref == -INFINITY ? 0.f : -mref;
          const uint64_t sl2x2 = f2(sl2, sl2), negref2 = f2(nref, nref);
          uint64_t acc2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            // The P pairs of keys [64 hh, 64 hh + 64) land in columns [32 hh,
            // 32 hh + 32), whose scores this or the previous half has loaded.
            uint32_t s0[32], s1[32], pk[32];
            tmem_ld32(sa + 64 * hh, s0);
            tmem_ld32(sa + 64 * hh + 32, s1);
            tmem_wait_ld_regs(s0);
            tmem_wait_ld_regs(s1);
            chunk_exp<false>(s0, sl2x2, negref2, acc2, pk);
            chunk_exp<false>(s1, sl2x2, negref2, acc2, pk + 16);
            tmem_st32(sa + 32 * hh, pk);
          }
          tmem_wait_st();
          float acc[4];
          f2_split(acc2[0], acc[0], acc[1]);
          f2_split(acc2[1], acc[2], acc[3]);
          l = l * alpha + ((acc[0] + acc[1]) + (acc[2] + acc[3]));
          if (__any_sync(0xffffffffu, rescale) && kc > kc0) {
            ok = wait_warp(&sh.pv_done[(kc - 1) % NS], (kc - 1) / NS);
            if (!ok) break;
            fence_after_sync();
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              const uint32_t oa = lane_base + TMEM_O + cc * 32;
              tmem_ld32(oa, o);
              tmem_wait_ld_regs(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(oa, o);
            }
            tmem_wait_st();
          }
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh.p_full[kc % NS]));
          ++kc;
        }
        if (ok && kc > kc0) ok = wait_warp(&sh.pv_done[(kc - 1) % NS], (kc - 1) / NS);
        // No kept block: O was never written.
        sh.sum[r] = kc > kc0 ? l : 0.f;
        sh.ref[r] = mref;
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh.l_full[it & 1]));
      }

      // ---- epilogue: deciders take O columns [0,64), exponential warps [64,128)
      if (ok) ok = wait_warp(&sh.l_full[it & 1], it >> 1);
      if (ok) {
        fence_after_sync();
        const int tok = r / a.G, sp = SPLIT ? sh.sp[it & 1] : -1, rows = x.ntok * a.G;
        const int64_t orow = (int64_t)(x.tok0 + tok) * a.Hq + sh.hk[it & 1] * a.G + (r - tok * a.G);
        const int col0 = decider ? 0 : 64;
        const float lrow = sh.sum[r], lref = sh.ref[r];
        const bool none = lrow == 0.f;  // no key kept for this row: the accumulator may hold anything
        const float inv = none ? 0.f : 1.f / lrow;
        // The rows leave through 4 KB of the tile's queries a warp (no longer needed): a
        // lane's row in 16-byte pieces, then 128-byte runs of four rows an instruction.
        const uint32_t stage = base + P_Q + (it & 1) * TILE_BYTES + warp * 4096;
        auto put_row = [&](int piece, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
          st_shared_v4(stage + lane * 128 + ((piece ^ (lane & 7)) * 16), v0, v1, v2, v3);
        };
        auto store_rows = [&](uint8_t *out, int64_t row_bytes) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int l2 = i * 4 + (lane >> 3), piece = lane & 7;
            const int64_t at = __shfl_sync(0xffffffffu, orow, l2);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(stage + l2 * 128 + ((piece ^ (l2 & 7)) * 16))
                         : "memory");
            if (quarter * 32 + l2 < rows) *reinterpret_cast<uint4 *>(out + at * row_bytes + piece * 16) = v;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t o[32];
          const int col = col0 + cc * 32;
          tmem_ld32(lane_base + TMEM_O + col, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = none ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
          if (sp < 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              put_row(cc * 4 + q, pack_bf16x2(__uint_as_float(o[8 * q]), __uint_as_float(o[8 * q + 1])),
                      pack_bf16x2(__uint_as_float(o[8 * q + 2]), __uint_as_float(o[8 * q + 3])),
                      pack_bf16x2(__uint_as_float(o[8 * q + 4]), __uint_as_float(o[8 * q + 5])),
                      pack_bf16x2(__uint_as_float(o[8 * q + 6]), __uint_as_float(o[8 * q + 7])));
            if (cc == 1) store_rows((uint8_t *)a.o + col0 * 2, D * 2);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              put_row(q, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            store_rows((uint8_t *)(a.o_part + (int64_t)sp * D + col), (int64_t)a.n_splits * D * 4);
          }
        }
        if (valid && !decider) {
          (sp < 0 ? a.lse + orow : a.lse_part + orow * a.n_splits + sp)[0] =
              none ? -INFINITY : lref * kLn2 + logf(lrow);
          if (SPLIT && sp < 0) a.lse_part[orow * a.n_splits] = __uint_as_float(kWholeRow);
        }
      }
      fence_proxy_async_smem();  // the staged rows, before the next queries
      fence_before_sync();       // and this warp's reads of O
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh.tile_empty[it & 1]));
    }
  }

  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == WARP_MMA) {
    fence_after_sync();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Merge of the split partials: LSE = ln sum_s exp(LSE_s), O = sum_s
// exp(LSE_s - LSE) O_s, splits without a key (LSE_s = -inf, O_s not written)
// left out; a NaN in one of them is the row's.  A warp takes ROWS query heads of a
// token, one after the other, four columns a lane; rows behind the last sequence keep
// what they held.  One row a warp is quickest for a decode step; with many rows the
// search for the sequence, once a row, was half the merge (16 prompts of 1024 tokens,
// 32 heads: 325 us in all with four rows a warp, 365 with one).
constexpr int MERGE_WARPS = 4, MERGE_ROWS = 4;
template <int ROWS>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_kernel(const ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * MERGE_WARPS + (threadIdx.x >> 5), groups = (a.Hq + ROWS - 1) / ROWS;
  const unsigned tok = unit / groups, h0 = (unit - tok * groups) * ROWS;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are complete
  if (tok >= (unsigned)a.total) return;
  // A token outside every (valid) sequence has no partial.  The number of entries of
  // cu[1..n] that are <= tok, by 32 probes a round.
  int lo = 0, hi = a.n_seq;
  while (lo < hi) {
    const int step = (hi - lo) / 33 + 1, at = lo + (lane + 1) * step;
    const bool ge = at <= hi && __ldg(a.cu_seqlens + at) <= (int)tok;
    const int c = __popc(__ballot_sync(0xffffffffu, ge));
    lo += c * step;
    hi = min(hi, lo + step - 1);
  }
  if (lo >= a.n_seq) return;
  const int c0 = __ldg(a.cu_seqlens + lo), c1 = __ldg(a.cu_seqlens + lo + 1);
  if (c0 < 0 || c0 > (int)tok || c1 - c0 > a.max_chunk || c1 > a.total) return;
#pragma unroll 1
  for (unsigned h = h0; h < h0 + ROWS && h < (unsigned)a.Hq; ++h) {
    const int64_t row = (int64_t)tok * a.Hq + h;
    const float *ls = a.lse_part + row * a.n_splits;
    if (__float_as_uint(ls[0]) == kWholeRow) continue;
    float m = -INFINITY;
#pragma unroll 1
    for (int s = lane; s < a.n_splits; s += 32) m = max_nan(m, ls[s]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 *op = reinterpret_cast<const float4 *>(a.o_part + row * a.n_splits * D) + lane;
#pragma unroll 4
    for (int s = 0; s < a.n_splits; ++s) {
      const float x = ls[s];
      if (x == -INFINITY) continue;
      const float w = expf(x - m);
      const float4 v = op[s * (D / 4)];
      z += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    const float inv = m == -INFINITY ? 0.f : 1.f / z;
    reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.o + row * D)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0) a.lse[row] = m == -INFINITY ? -INFINITY : m + logf(z);
  }
}

// 4-D map over the rows of a bf16 page pool: (column, slot, head, page).
bool make_map_pages(CUtensorMap *m, const KvPages &p, const void *ptr) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {D * 2, (cuuint64_t)p.page_size * D * 2, (cuuint64_t)p.page_stride};
  const cuuint32_t box[4] = {64, (cuuint32_t)(p.page_size < BN ? p.page_size : BN), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q: (column, head, token), box 64 columns x G heads x `tokens` tokens.
bool make_map_q(CUtensorMap *m, const ChunkArgs &a, int tokens) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {D, (cuuint64_t)a.Hq, (cuuint64_t)a.total};
  const cuuint64_t strides[2] = {D * 2, (cuuint64_t)a.q_tok_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t tiles_bound(int n_seq, int total, int max_chunk, int TT) {
  const int64_t by_len = (int64_t)n_seq * ((max_chunk + TT - 1) / TT);
  const int64_t by_total = (int64_t)(total + TT - 1) / TT + n_seq;
  return by_len < by_total ? by_len : by_total;
}

template <int FMT, bool REP, bool PAIR>
cudaError_t launch_one(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                       const ChunkArgs &a, int q_tokens, unsigned grid, cudaStream_t s) {
  constexpr uint32_t smem = Layout<FMT, PAIR>::END + ((sizeof(Shared) + 15) / 16) * 16;
  cudaError_t e = cudaFuncSetAttribute(chunk_paged_kernel<FMT, REP, PAIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_paged_kernel<FMT, REP, PAIR><<<grid, Cfg<FMT>::WARPS * 32, smem, s>>>(mq, mk, mv, a, q_tokens);
  return cudaGetLastError();
}

template <bool SPLIT>
cudaError_t launch_prompt(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                          const ChunkArgs &a, int q_tokens, unsigned grid, cudaStream_t s) {
  constexpr uint32_t smem = P_END + ((sizeof(PromptShared) + 15) / 16) * 16;
  const cudaError_t e = cudaFuncSetAttribute(prompt_paged_kernel<SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prompt_paged_kernel<SPLIT><<<grid, P_WARPS * 32, smem, s>>>(mq, mk, mv, a, q_tokens);
  return cudaGetLastError();
}

// Splits of at most this many blocks take half an SM a CTA where there are more CTAs
// than SMs: 64 sequences of up to 300 tokens 24 us against 32, of up to 1000 42 and
// 48, of 4 new tokens on 300 in three splits 47 and 75; with 16 blocks a split 71 and
// 72 (83 and 71 with a threshold: values arrive later), with 52 blocks 368 and 329.
constexpr int PAIR_BLOCKS = 12;

template <int FMT>
cudaError_t launch_fmt(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                       const ChunkArgs &a, int q_tokens, unsigned units, cudaStream_t s) {
  if (a.G * q_tokens <= 32) {
    if constexpr (FMT == kKvBf16)
      if (units > 152 && a.bps <= PAIR_BLOCKS)
        return launch_one<FMT, true, true>(mq, mk, mv, a, q_tokens, units, s);
    return launch_one<FMT, true, false>(mq, mk, mv, a, q_tokens, units, s);
  }
  if constexpr (FMT == kKvBf16) {
    // CTAs that stay pay where there are more tiles than SMs and these are short:
    // whole prompts of 256 tokens (64 of them) 137 us against 209, of 1024 (16) 203
    // and 270, of 4096 (4) 479 and 529, of 8192 (2) 835 and 868; a chunk of 4096 on
    // 16384, a hundred blocks a tile, 697 and 671 (a loop over tiles costs the loop
    // over blocks some registers).
    const int64_t keys = (int64_t)a.max_kv - a.max_chunk / 2;  // of a middle tile
    const unsigned grid = units / a.n_splits;  // (a tile's splits go to one CTA)
    if (grid > 152 && keys < (int64_t)64 * BN * a.n_splits)
      return a.n_splits > 1 ? launch_prompt<true>(mq, mk, mv, a, q_tokens, grid, s)
                            : launch_prompt<false>(mq, mk, mv, a, q_tokens, grid, s);
  }
  return launch_one<FMT, false, false>(mq, mk, mv, a, q_tokens, units, s);
}

}  // namespace

// The split count that a host-side model of the launch finds cheapest: waves of
// CTAs (one an SM, or two of the decode kernel), each a set-up and its share of
// the blocks, and the merge, a second launch (one sequence of 1000 tokens, bf16: 14.4
// us without it and 12.0 in eight splits where the calls are captured in a graph, 18
// and 23 where the host makes them one after another; the count is for the latter,
// and goes from 1 to 9 behind 1024 tokens).  A long decode batch takes six at least:
// sequences of different lengths fill the chip only in smaller pieces (24 sequences
// of 8192 to 32768 tokens, bf16: 295 us with 1 split, 288 with 3, 280 with 6, 303
// with 16).
int chunk_paged_splits(int n_seq, int total, int max_chunk, int max_kv, int Hkv, int TT, int format) {
  const int rows = (128 / TT) * (TT < max_chunk ? TT : max_chunk);
  const bool small = format != kKvBf16 && rows <= 8;
  const int slots = small ? 304 : 152;
  const int64_t units = tiles_bound(n_seq, total, max_chunk, TT) * Hkv;
  const int nb = (max_kv + BN - 1) / BN;
  // A block alone on its SM, and what it takes more on a full chip.
  const double block_us = format == kKvBf16 ? 0.65 : small ? 0.85 : 1.8;
  const double full_us = format == kKvBf16 ? 0.55 : small ? 0.65 : 0.0;
  const double setup_us = small ? 3.0 : 4.0, merge_us = 5.0;
  const int least = rows <= 32 && n_seq > 1 && nb >= 6 * 32 ? 6 : 1;
  int best = least;
  double best_t = 0;
  for (int n = least; n <= 64 && n <= (nb > 0 ? nb : 1); ++n) {
    const int bps = (nb + n - 1) / n;
    if (n > least && (nb + bps - 1) / bps < n) continue;  // the last splits would be empty
    const int64_t waves = (units * n + slots - 1) / slots;
    const double full = units * n < slots ? (double)(units * n) / slots : 1.0;
    const double t = waves * (setup_us + bps * (block_us + full * full_us)) + (n > 1 ? merge_us : 0);
    if (n == least || t < best_t) {
      best = n;
      best_t = t;
    }
  }
  return best;
}

// Bytes of the bf16 rows that a quantised cache is widened to first, 0 where it
// is not.  Widening a 128-key block of a KV head once moves about 100 KB (15 ns
// of the memory's time); converting it on the way costs each tile that reads it
// 0.7 us of an SM, 5 ns of the chip, so from three tiles of a sequence on the
// rows are written out (E4M3, 32 heads on 8: a chunk of 4096 on 16384, 1351 us
// with converters and 677 with widened rows; 16 chunks of 96 on 8192, 341 and 298;
// of 64, 227 and 249.  NVFP4: 1467 and 679, 367 and 301, 246 and 251).  Not where
// they would take over 4 GiB: the bound is the longest sequence's, for every
// sequence.
size_t chunk_paged_kv_bytes(int n_seq, int max_chunk, int max_kv, int Hkv, int TT, int format) {
  if (format == kKvBf16 || (max_chunk + TT - 1) / TT < 3) return 0;
  const size_t rows = (size_t)n_seq * Hkv * (((size_t)max_kv + BN - 1) / BN * BN);
  return rows * D * 2 * 2 <= (size_t)4 << 30 ? rows * D * 2 * 2 : 0;
}

cudaError_t launch_chunk_paged(const ChunkArgs &args, cudaStream_t s) {
  ChunkArgs a = args;
  if (a.kv_work) {
    const size_t bytes = chunk_paged_kv_bytes(a.n_seq, a.max_chunk, a.max_kv, a.Hkv, a.TT, a.pages.format);
    if (bytes && (int64_t)a.n_seq * a.Hkv <= 65535) {
      KvWidenArgs w{};
      w.pages = a.pages;
      w.k_out = a.kv_work;
      w.v_out = (char *)a.kv_work + bytes / 2;
      w.n_seq = a.n_seq; w.max_kv = a.max_kv; w.max_pages = a.max_pages;
      w.stride = (a.max_kv + BN - 1) / BN * BN;
      w.kv_len = a.kv_len; w.page_table = a.page_table; w.err = a.err;
      const cudaError_t e = launch_kv_widen(w, s);
      if (e != cudaSuccess) return e;
      KvPages &p = a.pages;  // from here on a bf16 cache of one page a sequence
      p.format = kKvBf16;
      p.k = w.k_out; p.v = w.v_out;
      p.n_pages = a.n_seq; p.page_size = w.stride; p.page_shift = -1;
      p.page_stride = (int64_t)a.Hkv * w.stride * D * 2;
      a.page_table = nullptr;
    }
  }
  const int64_t units = tiles_bound(a.n_seq, a.total, a.max_chunk, a.TT) * a.Hkv * a.n_splits;
  if (units > 0x7fffffffL) return cudaErrorNotYetImplemented;  // more CTAs than a grid has
  const int q_tokens = a.TT < a.max_chunk ? a.TT : a.max_chunk;
  if (a.bits) {  // words of tiles that a sequence does not have, and of untraversed blocks
    const cudaError_t e = cudaMemsetAsync(
        a.bits, 0, (size_t)a.n_seq * a.Hkv * a.n_t * a.n_splits * a.words * 4, s);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)units;
  cudaError_t e;
  if (a.pages.format != kKvBf16 && a.G * q_tokens <= 8) {
    e = launch_decode_paged(a, grid, s);
  } else {
    CUtensorMap mq, mk{}, mv{};
    if (!make_map_q(&mq, a, q_tokens)) return cudaErrorInvalidValue;
    if (a.pages.format == kKvBf16 &&
        (!make_map_pages(&mk, a.pages, a.pages.k) || !make_map_pages(&mv, a.pages, a.pages.v)))
      return cudaErrorInvalidValue;
    e = a.pages.format == kKvBf16   ? launch_fmt<kKvBf16>(mq, mk, mv, a, q_tokens, grid, s)
        : a.pages.format == kKvE4m3 ? launch_fmt<kKvE4m3>(mq, mk, mv, a, q_tokens, grid, s)
                                    : launch_fmt<kKvNvfp4>(mq, mk, mv, a, q_tokens, grid, s);
  }
  if (e != cudaSuccess || a.n_splits == 1) return e;
  // Several rows a warp once there are more than the chip's warps.
  const bool many = (int64_t)a.total * a.Hq > 152 * 64;
  const int per = many ? MERGE_ROWS : 1;
  const int64_t warps = (int64_t)a.total * ((a.Hq + per - 1) / per);
  // Launched as a programmatic dependent of the attention kernel, whose CTAs
  // release it as they start: its own launch is over by the time they end.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((warps + MERGE_WARPS - 1) / MERGE_WARPS));
  cfg.blockDim = dim3(MERGE_WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many ? merge_kernel<MERGE_ROWS> : merge_kernel<1>, a);
}

}  // namespace attn_skip
