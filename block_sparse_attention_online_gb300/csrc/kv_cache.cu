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
// Both kernels only move bytes: DRAM traffic bounds the large calls, latency
// the small ones.  Sixteen lanes own a row (16 bytes of bf16 each), so every
// row is read and written as whole 32-byte sectors and the row's maximum is
// four shuffles; a half warp takes kRows consecutive tokens of one head, whose
// pool rows are contiguous within a page, with all loads issued first.
#include <cuda_bf16.h>
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
  int64_t row;  // (page * Hkv + head) * page_size + slot: the row's scale index
  int64_t byte; // the row's first byte in k and v
  int ok;       // 0: no such row (out of range: reported by the caller)
};

template <int ROW_BYTES>
__device__ __forceinline__ Place place_of(const KvPages &p, const int32_t *table, int max_pages,
                                          int s, int64_t pos, int h) {
  Place x{0, 0, 0};
  const int64_t pi = pos / p.page_size;
  const int slot = (int)(pos - pi * p.page_size);
  if (pos < 0 || pi >= max_pages) return x;
  const int page = __ldg(table + (int64_t)s * max_pages + pi);
  if (page < 0 || page >= p.n_pages) return x;
  x.row = ((int64_t)page * p.Hkv + h) * p.page_size + slot;
  x.byte = (int64_t)page * p.page_stride + ((int64_t)h * p.page_size + slot) * ROW_BYTES;
  x.ok = 1;
  return x;
}

template <int FMT> struct RowBytes {
  static constexpr int value = FMT == kKvBf16 ? 2 * D : FMT == kKvE4m3 ? D : D / 2;
};

__device__ __forceinline__ float half_max(float m, unsigned hmask) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(hmask, m, o));
  return m;
}

// 2^i for i in [-126, 127].
__device__ __forceinline__ float pow2i(int i) { return __int_as_float((i + 127) << 23); }

// Smallest e with a <= top * 2^e for a > 0, top = 1.F * 2^TE (fraction bits TF).
template <int TE, int TF>
__device__ __forceinline__ int scale_exponent(float a) {
  int b = __float_as_int(a), ex = b >> 23;
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

// Eight elements of a new row (this lane's share) as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void *src, int64_t elem, float (&x)[8]) {
  if constexpr (F32) {
    const float4 *p = reinterpret_cast<const float4 *>((const float *)src + elem);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)src + elem));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int FMT>
__device__ __forceinline__ void store_row(const KvPages &p, bool value, const Place &at,
                                          const float (&x)[8], int hl, unsigned hmask) {
  uint8_t *codes = (uint8_t *)(value ? p.v : p.k) + at.byte;
  if constexpr (FMT == kKvBf16) {
    if (at.ok)
      *reinterpret_cast<uint4 *>(codes + hl * 16) =
          make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
    return;
  }
  float m = 0.f;
  bool fin = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmaxf(m, fabsf(x[i]));
    fin = fin && isfinite(x[i]);
  }
  const bool bad = (__ballot_sync(hmask, !fin) & hmask) != 0u;
  const float amax = half_max(m, hmask);
  // top = 448 = 1.75 * 2^8, or 2688 = 1.3125 * 2^11.
  const int e = bad || !(amax > 0.f) ? 0
                : FMT == kKvE4m3     ? scale_exponent<8, 0x600000>(amax)
                                     : scale_exponent<11, 0x280000>(amax);
  const float inv = pow2i(-e);
  uint8_t *scale = (value ? p.v_scale : p.k_scale) + at.row;
  if (at.ok && hl == 0) *scale = bad ? 255 : (uint8_t)(e + 127);
  if constexpr (FMT == kKvE4m3) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
    if (at.ok)
      *reinterpret_cast<uint2 *>(codes + hl * 8) =
          bad ? make_uint2(0, 0) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  } else {
    // Two lanes share a block of sixteen.
    const float bmax = fmaxf(m, __shfl_xor_sync(hmask, m, 1)) * inv;
    // Nearest E4M3 to bmax / 6, then one code up if it lies below.
    uint32_t b = e4m3x2(__fdiv_rn(bmax, 6.f), 0.f) & 0xffu;
    if (6.f * e4m3_value(b) < bmax) ++b;
    const float s = e4m3_value(b), by = s > 0.f ? s : 1.f;  // b = 0 only for sixteen zeros
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // y / s in fp32 rounds to an E2M1 midpoint only when it is one: a
      // midpoint times s has at most 7 significant bits, so y either equals it
      // or is at least one fp32 step away from it.
      w |= e2m1x2(__fdiv_rn(x[2 * i] * inv, by), __fdiv_rn(x[2 * i + 1] * inv, by)) << (8 * i);
    }
    if (at.ok) {
      *reinterpret_cast<uint32_t *>(codes + hl * 4) = bad ? 0u : w;
      if ((hl & 1) == 0) (value ? p.v_bs : p.k_bs)[at.row * (D / 16) + (hl >> 1)] = bad ? 0 : b;
    }
  }
}

// One half warp: kRows consecutive tokens of one (head, key or value).
template <int FMT, bool F32, int kRows>
__global__ void __launch_bounds__(NT) kv_append_kernel(const KvAppendArgs a) {
  const int hl = threadIdx.x & 15;
  const unsigned hmask = 0xffffu << (threadIdx.x & 16);
  const int64_t unit = (int64_t)blockIdx.x * HALVES + (threadIdx.x >> 4);
  const int per = 2 * a.pages.Hkv;
  const int64_t t0 = unit / per * kRows;
  if (t0 >= a.total) return;
  const int hv = (int)(unit % per);
  const bool value = hv >= a.pages.Hkv;
  const int h = value ? hv - a.pages.Hkv : hv;
  const void *src = value ? a.v_new : a.k_new;
  const int64_t ts = value ? a.v_tok_stride : a.k_tok_stride;
  float x[kRows][8];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (t0 + r < a.total) load8<F32>(src, (t0 + r) * ts + (int64_t)h * D + hl * 8, x[r]);
  int s = find_seq(a.cu_seqlens, a.n_seq, (int)t0, hl, hmask);
  Place at[kRows];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    at[r].ok = 0;
    const int t = (int)t0 + r;
    while (s < a.n_seq && __ldg(a.cu_seqlens + s + 1) <= t) ++s;
    if (t >= a.total || s >= a.n_seq) continue;  // behind the last sequence
    const int c0 = __ldg(a.cu_seqlens + s), c1 = __ldg(a.cu_seqlens + s + 1);
    const int len = __ldg(a.kv_len + s);
    // The sequence's bounds and its length are checked as a whole, so that no
    // row of a sequence with a bad length is written.
    if (c0 < 0 || c0 > t || c1 > a.total || len < 0 ||
        len > (int64_t)a.max_pages * a.pages.page_size) {
      bad = true;
      continue;
    }
    const int64_t pos = (int64_t)len - c1 + t;
    if (pos < 0) continue;  // the chunk is longer than the cache: no such position
    at[r] = place_of<RowBytes<FMT>::value>(a.pages, a.page_table, a.max_pages, s, pos, h);
    bad |= !at[r].ok;
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (t0 + r < a.total) store_row<FMT>(a.pages, value, at[r], x[r], hl, hmask);
  }
  if (bad && hl == 0) atomicOr(a.err, kErrBadArg);
}

// This lane's eight elements of a stored row as fp32 (exact).
struct Raw {
  uint4 c;       // codes
  uint32_t s, b; // row scale byte, block scale byte
};

template <int FMT>
__device__ __forceinline__ Raw load_raw(const KvPages &p, bool value, const Place &at, int hl) {
  Raw r{make_uint4(0, 0, 0, 0), 127, 0};
  if (!at.ok) return r;
  const uint8_t *codes = (const uint8_t *)(value ? p.v : p.k) + at.byte;
  if constexpr (FMT == kKvBf16) {
    r.c = __ldg(reinterpret_cast<const uint4 *>(codes + hl * 16));
  } else {
    r.s = __ldg((value ? p.v_scale : p.k_scale) + at.row);
    if constexpr (FMT == kKvE4m3) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(codes + hl * 8));
      r.c.x = v.x;
      r.c.y = v.y;
    } else {
      r.c.x = __ldg(reinterpret_cast<const uint32_t *>(codes + hl * 4));
      r.b = __ldg((value ? p.v_bs : p.k_bs) + at.row * (D / 16) + (hl >> 1));
    }
  }
  return r;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float f, float &lo, float &hi) {
  lo = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu))) * f;
  hi = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * f;
}

template <int FMT>
__device__ __forceinline__ void decode_raw(const Raw &r, float (&x)[8]) {
  if constexpr (FMT == kKvBf16) {
    const uint32_t w[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return;
  }
  // Byte 0 stands for 2^-127 (an fp32 subnormal), 255 for NaN.
  const float f = r.s == 255u ? NAN : r.s == 0u ? 5.877471754111438e-39f : __uint_as_float(r.s << 23);
  if constexpr (FMT == kKvE4m3) {
    const uint32_t w[2] = {r.c.x, r.c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
          : "=r"(h)
          : "h"((unsigned short)(w[i >> 1] >> (16 * (i & 1)))));
      f16x2_to_f32(h, f, x[2 * i], x[2 * i + 1]);
    }
  } else {
    const float s = e4m3_value(r.b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
          : "=r"(h)
          : "r"((r.c.x >> (8 * i)) & 0xffu));
      f16x2_to_f32(h, s, x[2 * i], x[2 * i + 1]);  // exact: at most six bits
      x[2 * i] *= f;
      x[2 * i + 1] *= f;
    }
  }
}

template <int FMT, bool F32, int kRows>
__global__ void __launch_bounds__(NT) kv_gather_kernel(const KvGatherArgs a) {
  const int hl = threadIdx.x & 15;
  const unsigned hmask = 0xffffu << (threadIdx.x & 16);
  const int64_t unit = (int64_t)blockIdx.x * HALVES + (threadIdx.x >> 4);
  const int per = 2 * a.pages.Hkv;
  const int64_t t0 = unit / per * kRows;
  if (t0 >= a.total) return;
  const int hv = (int)(unit % per);
  const bool value = hv >= a.pages.Hkv;
  const int h = value ? hv - a.pages.Hkv : hv;
  int s = find_seq(a.cu_rows, a.n_seq, (int)t0, hl, hmask);
  Place at[kRows];
  Raw raw[kRows];
  bool bad = false, write[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int t = (int)t0 + r;
    at[r].ok = 0;
    write[r] = false;
    while (s < a.n_seq && __ldg(a.cu_rows + s + 1) <= t) ++s;
    if (t >= a.total || s >= a.n_seq) continue;
    const int c0 = __ldg(a.cu_rows + s);
    write[r] = true;
    if (c0 >= 0 && c0 <= t) {
      const int64_t pos = (int64_t)(a.start ? __ldg(a.start + s) : 0) + (t - c0);
      at[r] = place_of<RowBytes<FMT>::value>(a.pages, a.page_table, a.max_pages, s, pos, h);
    }
    bad |= !at[r].ok;
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) raw[r] = load_raw<FMT>(a.pages, value, at[r], hl);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (!write[r]) continue;
    float x[8];
    decode_raw<FMT>(raw[r], x);
    const int64_t elem = ((t0 + r) * a.pages.Hkv + h) * D + hl * 8;
    if constexpr (F32) {
      float4 *o = reinterpret_cast<float4 *>((float *)(value ? a.v_out : a.k_out) + elem);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4 *>((__nv_bfloat16 *)(value ? a.v_out : a.k_out) + elem) =
          make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
    }
  }
  if (bad && hl == 0) atomicOr(a.err, kErrBadArg);
}

// Rows per half warp: four when that still gives every SM a full set of
// blocks, else one, so that a small call spreads over the chip.
constexpr int kManyRows = 4;
bool many_rows(int64_t total, int Hkv) {
  return total * 2 * Hkv >= (int64_t)kManyRows * HALVES * 152 * 8;
}
unsigned grid_of(int64_t total, int Hkv, int rows) {
  const int64_t units = (total + rows - 1) / rows * 2 * Hkv;
  return (unsigned)((units + HALVES - 1) / HALVES);
}

template <int FMT, bool F32>
void append_fmt(const KvAppendArgs &a, cudaStream_t s) {
  if (many_rows(a.total, a.pages.Hkv))
    kv_append_kernel<FMT, F32, kManyRows><<<grid_of(a.total, a.pages.Hkv, kManyRows), NT, 0, s>>>(a);
  else
    kv_append_kernel<FMT, F32, 1><<<grid_of(a.total, a.pages.Hkv, 1), NT, 0, s>>>(a);
}
template <int FMT, bool F32>
void gather_fmt(const KvGatherArgs &a, cudaStream_t s) {
  if (many_rows(a.total, a.pages.Hkv))
    kv_gather_kernel<FMT, F32, kManyRows><<<grid_of(a.total, a.pages.Hkv, kManyRows), NT, 0, s>>>(a);
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

}  // namespace attn_skip
