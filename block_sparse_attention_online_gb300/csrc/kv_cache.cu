// The paged key/value cache: new rows written to its pages (quantised on the
// way for the E4M3 and NVFP4 formats) and rows read back.
//
// A row is the 128 elements of one (token, KV head).  With x the row in fp32:
//   scale   2^e, the smallest power of two with max|x| <= top * 2^e, where top
//           is the largest value the codes reach (448 for E4M3, 6 * 448 for
//           NVFP4), e clamped to [-110, 120] and stored as the byte e + 127;
//           a zero row has e = 0; a row with an infinity or a NaN is stored as
//           byte 255 and reads back as NaN;
//   E4M3    code = x / 2^e rounded to nearest even (the division is exact);
//   NVFP4   y = x / 2^e; per 16 elements b = the smallest E4M3 value with
//           6 b >= max|y|; code = E2M1(y / b) rounded to nearest even.
// With a power of two as the row scale a stored element has at most 4 (E4M3)
// or 6 (E2M1 times E4M3) significant bits, so reading back in bf16 is exact
// (e >= -110 keeps the smallest product, 2^-10 * 2^-110, a bf16 normal).
//
// DRAM traffic bounds the large calls, instruction issue those that quantise (E4M3,
// 16384 tokens of 8 heads: 22 us, 15 for the bytes), latency the small ones.  Sixteen lanes own a row, so every row is read and written as
// whole 32-byte sectors and the row's maximum is four shuffles.  A half warp
// takes the key and the value rows of a few consecutive tokens of one head,
// whose place in the cache it works out once a token and whose pool rows are
// contiguous within a page; all its loads are issued first.
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include "internal.h"

namespace attn_skip {
namespace {

constexpr int D = 128;
constexpr int NT = 256;        // 16 half warps
constexpr int HALVES = NT / 16;
constexpr int EMIN = -110, EMAX = 120;

// The sequence of packed row t: the number of entries of cu[1..n] that are
// <= t, by a 17-way search with sixteen probes a round (one round of loads for
// up to 16 sequences, two for up to 288).  n_seq when t lies behind the last.
__device__ __forceinline__ int find_seq(const int32_t *cu, int n, int t, int hl, unsigned hmask) {
  int lo = 0, hi = n;  // answer in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo) / 17 + 1;  // 17 steps reach past hi
    const int p = lo + (hl + 1) * step;  // probe cu[p]: is row t at or behind it?
    const bool ge = p <= hi && __ldg(cu + p) <= t;
    const int c = __popc(__ballot_sync(hmask, ge) & hmask);
    const int nlo = lo + c * step;
    hi = min(hi, nlo + step - 1);
    lo = nlo;
  }
  return lo;
}

struct Place {
  int64_t row;  // (page * Hkv + head) * page_size + slot: the rows' scale index
  int64_t byte; // the rows' first byte in k and v
  int left;     // rows of the page from this one on; 0: no such rows
  __device__ __forceinline__ bool ok() const { return left > 0; }
};

// Rows of position pos of sequence s, head h.
template <int ROW_BYTES>
__device__ __forceinline__ Place place_of(const KvPages &p, const int32_t *table, int max_pages,
                                          int s, int64_t pos, int h) {
  Place x{0, 0, 0};
  if (pos < 0 || pos >= (int64_t)max_pages * p.page_size) return x;
  const unsigned u = (unsigned)pos;
  const unsigned pi = p.page_shift >= 0 ? u >> p.page_shift : u / (unsigned)p.page_size;
  const int slot = (int)(u - pi * (unsigned)p.page_size);
  const int page = __ldg(table + (int64_t)s * max_pages + pi);
  if (page < 0 || page >= p.n_pages) return x;
  const int in_page = h * p.page_size + slot;
  x.row = (int64_t)page * (p.Hkv * p.page_size) + in_page;
  x.byte = (int64_t)page * p.page_stride + (int64_t)in_page * ROW_BYTES;
  x.left = p.page_size - slot;
  return x;
}

// The next position's: the next row of the page, or a page to look up.
template <int ROW_BYTES>
__device__ __forceinline__ Place next_place(const Place &at, const KvPages &p, const int32_t *table,
                                            int max_pages, int s, int64_t pos, int h) {
  if (at.left > 1) return Place{at.row + 1, at.byte + ROW_BYTES, at.left - 1};
  return place_of<ROW_BYTES>(p, table, max_pages, s, pos, h);
}

template <int FMT> struct RowBytes {
  static constexpr int value = FMT == kKvBf16 ? 2 * D : FMT == kKvE4m3 ? D : D / 2;
};

// 2^i for i in [-126, 127].
__device__ __forceinline__ float pow2i(int i) { return __int_as_float((i + 127) << 23); }

// Smallest e with a <= top * 2^e for the fp32 a > 0 of bits b, top = 1.F * 2^TE
// (fraction bits TF), clamped.
template <int TE, int TF>
__device__ __forceinline__ int scale_exponent(uint32_t b) {
  const int ex = (int)(b >> 23);
  if (ex == 0) return EMIN;  // fp32 subnormal: far below the clamp
  return min(EMAX, max(EMIN, ex - 127 - TE + ((b & 0x7fffff) > TF ? 1 : 0)));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {  // codes 0x00 to 0x7e
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)code));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// This lane's eight elements of a new row, as they come.
template <bool F32> struct New;
template <> struct New<false> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void *src, int64_t elem) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)src + elem));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // Bits of the largest |element| (fp32; infinities and NaN compare above all).
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t x = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
    return max(x << 16, x & 0xffff0000u);
  }
};
template <> struct New<true> {
  float x[8];
  __device__ __forceinline__ void load(const void *src, int64_t elem) {
    const float4 *p = reinterpret_cast<const float4 *>((const float *)src + elem);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ float at(int i) const { return x[i]; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Largest |element| of a token's key row and value row (fp32 bits), over the
// row's sixteen lanes, and over this lane and its neighbour (a block of sixteen).
struct Tops {
  uint32_t row[2], pair[2];
};
template <bool F32>
__device__ __forceinline__ Tops tops_of(const New<F32> &k, const New<F32> &v, unsigned hmask) {
  Tops t;
  if constexpr (F32) {
    t.row[0] = k.top();
    t.row[1] = v.top();
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        t.row[w] = max(t.row[w], __shfl_xor_sync(hmask, t.row[w], o));
        if (o == 1) t.pair[w] = t.row[w];
      }
    }
  } else {  // both rows' as the halves of one word
    uint32_t m = (k.top() >> 16) | v.top();
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      m = __vmaxu2(m, __shfl_xor_sync(hmask, m, o));
      if (o == 1) {
        t.pair[0] = m << 16;
        t.pair[1] = m & 0xffff0000u;
      }
    }
    t.row[0] = m << 16;
    t.row[1] = m & 0xffff0000u;
  }
  return t;
}

// The row whose eight elements a lane holds is x, to its place; half warp.  m,
// pair: its tops.
template <int FMT, bool F32>
__device__ __forceinline__ void store_row(const KvPages &p, bool value, const Place &at,
                                          const New<F32> &x, uint32_t m, uint32_t pair, int hl) {
  uint8_t *codes = (uint8_t *)(value ? p.v : p.k) + at.byte;
  if constexpr (FMT == kKvBf16) {
    if (!at.ok()) return;
    uint4 v;
    if constexpr (F32)
      v = make_uint4(bf16x2(x.at(0), x.at(1)), bf16x2(x.at(2), x.at(3)), bf16x2(x.at(4), x.at(5)),
                     bf16x2(x.at(6), x.at(7)));
    else
      v = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    *reinterpret_cast<uint4 *>(codes + hl * 16) = v;
  } else {
    const bool bad = m >= 0x7f800000u;  // an infinity or a NaN
    // top = 448 = 1.75 * 2^8, or 2688 = 1.3125 * 2^11.
    const int e = bad || m == 0u     ? 0
                  : FMT == kKvE4m3 ? scale_exponent<8, 0x600000>(m)
                                   : scale_exponent<11, 0x280000>(m);
    const float inv = pow2i(-e);
    if (at.ok() && hl == 0) (value ? p.v_scale : p.k_scale)[at.row] = bad ? 255 : (uint8_t)(e + 127);
    if constexpr (FMT == kKvE4m3) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x.at(2 * i) * inv, x.at(2 * i + 1) * inv);
      if (at.ok())
        *reinterpret_cast<uint2 *>(codes + hl * 8) =
            bad ? make_uint2(0, 0) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    } else {
      // Two lanes share a block of sixteen.
      const float bmax = __uint_as_float(pair) * inv;
      // Nearest E4M3 to bmax / 6, then one code up if it lies below.
      uint32_t b = e4m3x2(__fdiv_rn(bmax, 6.f), 0.f) & 0xffu;
      if (6.f * e4m3_value(b) < bmax) ++b;
      const float s = e4m3_value(b), by = s > 0.f ? s : 1.f;  // b = 0 only for sixteen zeros
      uint32_t w = 0;
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // y / s in fp32 rounds to an E2M1 midpoint only when it is one: a
          // midpoint times s has at most 7 significant bits, so y either equals it
          // or is at least one fp32 step away from it.
          w |= e2m1x2(__fdiv_rn(x.at(2 * i) * inv, by), __fdiv_rn(x.at(2 * i + 1) * inv, by)) << (8 * i);
        }
      } else {
        // bf16 elements: a y that is no midpoint times s is 2^-8 of it away, so a
        // product with 1 / s, at most two fp32 steps off, decides, once it is moved
        // four steps to the side to which a tie goes (the even code): up where the
        // fraction is 1.5 or more (0.75, 1.75, 3.5), down where it is less (0.25,
        // 1.25, 2.5, 5).  Against a division an element:
        // 16384 rows in 34 us, not 38.
        const float r = inv * __frcp_rn(by);
        auto near = [&](float v) {
          const float q = v * r;
          const uint32_t b = __float_as_uint(q);
          return fabsf(q) < 0.125f ? q : __uint_as_float(b + ((b >> 19) & 8u) - 4u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w |= e2m1x2(near(x.at(2 * i)), near(x.at(2 * i + 1))) << (8 * i);
      }
      if (at.ok()) {
        *reinterpret_cast<uint32_t *>(codes + hl * 4) = bad ? 0u : w;
        if ((hl & 1) == 0) (value ? p.v_bs : p.k_bs)[at.row * (D / 16) + (hl >> 1)] = bad ? 0 : b;
      }
    }
  }
}

// The last block of a call reports every sequence with bad bounds, whether or not a
// row of the call falls into it (the others leave its rows out).  (The loop unrolled
// makes the call's other blocks slower: 16384 tokens into E4M3 pages 24.6 us, 22.1.)
__device__ __forceinline__ void check_bounds(const int32_t *cu, int n, int total, unsigned *err) {
  bool bad = false;
#pragma unroll 1
  for (int s = threadIdx.x; s < n; s += NT) {
    const int c0 = __ldg(cu + s), c1 = __ldg(cu + s + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > total;
  }
  if (bad) atomicOr(err, kErrBadArg);
}

// One half warp: the key and value rows of kTok consecutive tokens of one head.
template <int FMT, bool F32, int kTok>
__global__ void __launch_bounds__(NT) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  const int hl = threadIdx.x & 15;
  const unsigned hmask = 0xffffu << (threadIdx.x & 16);
  const unsigned unit = blockIdx.x * HALVES + (threadIdx.x >> 4);
  const unsigned tg = unit / (unsigned)a.pages.Hkv;
  const int h = (int)(unit - tg * (unsigned)a.pages.Hkv);
  const int64_t t0 = (int64_t)tg * kTok;
  if (t0 >= a.total) {
    if (blockIdx.x == gridDim.x - 1) check_bounds(a.cu_seqlens, a.n_seq, a.total, a.err);
    return;
  }
  New<F32> x[kTok][2];
#pragma unroll
  for (int r = 0; r < kTok; ++r)
    if (t0 + r < a.total) {
      x[r][0].load(a.k_new, (t0 + r) * a.k_tok_stride + h * D + hl * 8);
      x[r][1].load(a.v_new, (t0 + r) * a.v_tok_stride + h * D + hl * 8);
    }
  int s = find_seq(a.cu_seqlens, a.n_seq, (int)t0, hl, hmask) - 1;
  bool bad = false;
  int end = INT_MIN;    // the current sequence's last row + 1
  int first = INT_MAX;  // its first row that has a position
  int64_t shift = 0;    // position minus row
  Place at{0, 0, 0};
#pragma unroll
  for (int r = 0; r < kTok; ++r) {
    const int t = (int)t0 + r;
    if (t >= a.total) break;
    if (t >= end) {  // the next sequence that has rows
      do {
        ++s;
      } while (s < a.n_seq && __ldg(a.cu_seqlens + s + 1) <= t);
      if (s >= a.n_seq) break;  // behind the last sequence
      const int c0 = __ldg(a.cu_seqlens + s), len = __ldg(a.kv_len + s);
      end = __ldg(a.cu_seqlens + s + 1);
      shift = (int64_t)len - end;
      // The sequence's bounds and its length are checked as a whole, so that no
      // row of a sequence with a bad length is written.
      const bool fine = c0 >= 0 && c0 <= end && end <= a.total && len >= 0 &&
                        len <= (int64_t)a.max_pages * a.pages.page_size;
      bad |= !fine;
      at.left = 0;
      // (A chunk may be longer than its cache: rows before position 0 have no place.
      // Nor have rows before the first sequence.)
      first = fine ? max(c0, end - len) : INT_MAX;
    }
    if (t >= first) {
      at = next_place<RowBytes<FMT>::value>(at, a.pages, a.page_table, a.max_pages, s, shift + t, h);
      bad |= !at.ok();
    }
    Tops m{};
    if constexpr (FMT != kKvBf16) m = tops_of<F32>(x[r][0], x[r][1], hmask);
    store_row<FMT, F32>(a.pages, false, at, x[r][0], m.row[0], m.pair[0], hl);
    store_row<FMT, F32>(a.pages, true, at, x[r][1], m.row[1], m.pair[1], hl);
  }
  if (bad && hl == 0) atomicOr(a.err, kErrBadArg);
}

// This lane's share of a stored row: two runs of four elements, for which the
// outputs' 16-byte (fp32) or 8-byte (bf16) stores are contiguous over the lanes.
// Run i: elements 64 i + 4 hl and on.
struct Raw {
  uint2 c[2];     // codes (bf16: the elements)
  uint32_t s;     // row scale byte
  uint32_t b[2];  // block scale bytes
};

template <int FMT>
__device__ __forceinline__ Raw load_raw(const KvPages &p, bool value, const Place &at, int hl) {
  Raw r{{make_uint2(0, 0), make_uint2(0, 0)}, 127, {0, 0}};
  if (!at.ok()) return r;
  const uint8_t *codes = (const uint8_t *)(value ? p.v : p.k) + at.byte;
  if constexpr (FMT != kKvBf16) r.s = __ldg((value ? p.v_scale : p.k_scale) + at.row);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (FMT == kKvBf16) {
      r.c[i] = __ldg(reinterpret_cast<const uint2 *>(codes + i * 128) + hl);
    } else if constexpr (FMT == kKvE4m3) {
      r.c[i].x = __ldg(reinterpret_cast<const uint32_t *>(codes + i * 64) + hl);
    } else {
      r.c[i].x = __ldg(reinterpret_cast<const uint16_t *>(codes + i * 32) + hl);
      r.b[i] = __ldg((value ? p.v_bs : p.k_bs) + at.row * (D / 16) + i * 4 + (hl >> 2));
    }
  }
  return r;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float f, float &lo, float &hi) {
  lo = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu))) * f;
  hi = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * f;
}

// Byte 0 stands for 2^-127 (an fp32 subnormal), 255 for NaN.
__device__ __forceinline__ float row_scale(uint32_t byte) {
  return byte == 255u ? NAN : byte == 0u ? 5.877471754111438e-39f : __uint_as_float(byte << 23);
}

// Run i as fp32 (exact).
template <int FMT>
__device__ __forceinline__ void decode_raw(const Raw &r, int i, float f, float (&x)[4]) {
  if constexpr (FMT == kKvBf16) {
    x[0] = __uint_as_float(r.c[i].x << 16);
    x[1] = __uint_as_float(r.c[i].x & 0xffff0000u);
    x[2] = __uint_as_float(r.c[i].y << 16);
    x[3] = __uint_as_float(r.c[i].y & 0xffff0000u);
  } else {
    uint32_t h[2];
    if constexpr (FMT == kKvE4m3) {
      asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
          "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
          : "=r"(h[0]), "=r"(h[1])
          : "r"(r.c[i].x));
      f16x2_to_f32(h[0], f, x[0], x[1]);
      f16x2_to_f32(h[1], f, x[2], x[3]);
    } else {
      asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
          : "=r"(h[0]), "=r"(h[1])
          : "r"(r.c[i].x));
      const float s = e4m3_value(r.b[i]);  // code times block scale: exact, at most six bits
      f16x2_to_f32(h[0], s, x[0], x[1]);
      f16x2_to_f32(h[1], s, x[2], x[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= f;
    }
  }
}

template <int FMT, bool F32, int kTok>
__global__ void __launch_bounds__(NT) kv_gather_kernel(const __grid_constant__ KvGatherArgs a) {
  const int hl = threadIdx.x & 15;
  const unsigned hmask = 0xffffu << (threadIdx.x & 16);
  const unsigned unit = blockIdx.x * HALVES + (threadIdx.x >> 4);
  const unsigned tg = unit / (unsigned)a.pages.Hkv;
  const int h = (int)(unit - tg * (unsigned)a.pages.Hkv);
  const int64_t t0 = (int64_t)tg * kTok;
  if (t0 >= a.total) {
    if (blockIdx.x == gridDim.x - 1) check_bounds(a.cu_rows, a.n_seq, a.total, a.err);
    return;
  }
  int s = find_seq(a.cu_rows, a.n_seq, (int)t0, hl, hmask) - 1;
  Raw raw[kTok][2];
  bool bad = false, fine = false;
  unsigned mine = 0;  // rows of sequences (the others stay as they were)
  int c0 = 0, end = INT_MIN;
  int64_t shift = 0;  // position minus row
  Place at{0, 0, 0};
#pragma unroll
  for (int r = 0; r < kTok; ++r) {
    const int t = (int)t0 + r;
    if (t >= a.total) break;
    if (t >= end) {  // the next sequence that has rows
      do {
        ++s;
      } while (s < a.n_seq && __ldg(a.cu_rows + s + 1) <= t);
      if (s >= a.n_seq) break;
      c0 = __ldg(a.cu_rows + s);
      end = __ldg(a.cu_rows + s + 1);
      shift = (int64_t)(a.start ? __ldg(a.start + s) : 0) - c0;
      fine = c0 >= 0 && c0 <= end && end <= a.total;
      at.left = 0;
    }
    if (fine && t < c0) continue;  // before the first sequence
    mine |= 1u << r;
    if (fine)
      at = next_place<RowBytes<FMT>::value>(at, a.pages, a.page_table, a.max_pages, s, shift + t, h);
    bad |= !at.ok();
    raw[r][0] = load_raw<FMT>(a.pages, false, at, hl);
    raw[r][1] = load_raw<FMT>(a.pages, true, at, hl);
  }
#pragma unroll
  for (int r = 0; r < kTok; ++r) {
    if (!(mine >> r & 1u)) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const Raw &y = raw[r][w];
      const float f = row_scale(y.s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x[4];
        decode_raw<FMT>(y, i, f, x);
        const int64_t elem = ((t0 + r) * a.pages.Hkv + h) * D + i * 64 + hl * 4;
        void *out = w ? a.v_out : a.k_out;
        if constexpr (F32)
          *reinterpret_cast<float4 *>((float *)out + elem) = make_float4(x[0], x[1], x[2], x[3]);
        else
          *reinterpret_cast<uint2 *>((__nv_bfloat16 *)out + elem) =
              make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
      }
    }
  }
  if (bad && hl == 0) atomicOr(a.err, kErrBadArg);
}

// Every cached row of a quantised cache as bf16 (exact), sequence s's head h at
// rows [(s * Hkv + h) * stride, ..) of k_out and v_out, for a bf16 kernel that
// reads them many times.  One half warp: the key and value rows of four
// consecutive positions of one (sequence, head).  A row of a page id out of range
// becomes zeros.
template <int FMT>
__global__ void __launch_bounds__(NT) kv_widen_kernel(const __grid_constant__ KvWidenArgs a) {
  constexpr int kTok = 4;
  const int hl = threadIdx.x & 15;
  const int p0 = (int)(blockIdx.x * HALVES + (threadIdx.x >> 4)) * kTok;
  const int h = (int)(blockIdx.y % (unsigned)a.pages.Hkv), s = (int)(blockIdx.y / (unsigned)a.pages.Hkv);
  int len = __ldg(a.kv_len + s);
  if (len > a.max_kv) len = 0;  // (a bad length is an empty cache; the attention reports it)
  if (p0 >= len) return;
  Raw raw[kTok][2];
  bool bad = false;
  Place at{0, 0, 0};
#pragma unroll
  for (int r = 0; r < kTok; ++r) {
    if (p0 + r >= len) break;
    at = next_place<RowBytes<FMT>::value>(at, a.pages, a.page_table, a.max_pages, s, p0 + r, h);
    bad |= !at.ok();
    raw[r][0] = load_raw<FMT>(a.pages, false, at, hl);
    raw[r][1] = load_raw<FMT>(a.pages, true, at, hl);
  }
  const int64_t row0 = ((int64_t)s * a.pages.Hkv + h) * a.stride + p0;
#pragma unroll
  for (int r = 0; r < kTok; ++r) {
    if (p0 + r >= len) break;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const Raw &y = raw[r][w];
      const float f = row_scale(y.s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x[4];
        decode_raw<FMT>(y, i, f, x);
        *reinterpret_cast<uint2 *>((__nv_bfloat16 *)(w ? a.v_out : a.k_out) + (row0 + r) * D + i * 64 + hl * 4) =
            make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
      }
    }
  }
  if (bad && hl == 0) atomicOr(a.err, kErrBadArg);
}

// Tokens per half warp: four (two of fp32 rows) when that still gives every SM
// eight blocks, else one, so that a small call spreads over the chip.
template <bool F32> constexpr int kMany = F32 ? 2 : 4;
bool many(int64_t total, int Hkv) { return total * Hkv >= (int64_t)4 * HALVES * 152 * 8; }
unsigned grid_of(int64_t total, int Hkv, int tok) {
  const int64_t units = (total + tok - 1) / tok * Hkv;
  return (unsigned)((units + HALVES - 1) / HALVES) + 1;  // and check_bounds'
}

template <int FMT, bool F32>
void append_fmt(const KvAppendArgs &a, cudaStream_t s) {
  constexpr int M = kMany<F32>;
  if (many(a.total, a.pages.Hkv))
    kv_append_kernel<FMT, F32, M><<<grid_of(a.total, a.pages.Hkv, M), NT, 0, s>>>(a);
  else
    kv_append_kernel<FMT, F32, 1><<<grid_of(a.total, a.pages.Hkv, 1), NT, 0, s>>>(a);
}
template <int FMT, bool F32>
void gather_fmt(const KvGatherArgs &a, cudaStream_t s) {
  constexpr int M = kMany<F32>;
  if (many(a.total, a.pages.Hkv))
    kv_gather_kernel<FMT, F32, M><<<grid_of(a.total, a.pages.Hkv, M), NT, 0, s>>>(a);
  else
    kv_gather_kernel<FMT, F32, 1><<<grid_of(a.total, a.pages.Hkv, 1), NT, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s) {
  switch (a.pages.format) {
    case kKvBf16: a.src_f32 ? append_fmt<kKvBf16, true>(a, s) : append_fmt<kKvBf16, false>(a, s); break;
    case kKvE4m3: a.src_f32 ? append_fmt<kKvE4m3, true>(a, s) : append_fmt<kKvE4m3, false>(a, s); break;
    default: a.src_f32 ? append_fmt<kKvNvfp4, true>(a, s) : append_fmt<kKvNvfp4, false>(a, s); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_gather(const KvGatherArgs &a, cudaStream_t s) {
  switch (a.pages.format) {
    case kKvBf16: a.out_f32 ? gather_fmt<kKvBf16, true>(a, s) : gather_fmt<kKvBf16, false>(a, s); break;
    case kKvE4m3: a.out_f32 ? gather_fmt<kKvE4m3, true>(a, s) : gather_fmt<kKvE4m3, false>(a, s); break;
    default: a.out_f32 ? gather_fmt<kKvNvfp4, true>(a, s) : gather_fmt<kKvNvfp4, false>(a, s); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_widen(const KvWidenArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.max_kv + 4 * HALVES - 1) / (4 * HALVES)),
                  (unsigned)(a.n_seq * a.pages.Hkv));
  if (a.pages.format == kKvE4m3)
    kv_widen_kernel<kKvE4m3><<<grid, NT, 0, s>>>(a);
  else
    kv_widen_kernel<kKvNvfp4><<<grid, NT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace attn_skip
