// Drafted tokens against the target's probabilities (speculative sampling).
//
// Drafted token i of a sequence, drawn from q_i, is accepted if u_i q_i(x_i) < p_i(x_i)
// and all before it are; at the first rejected one the token is drawn from the positive
// part of p_i - q_i instead (from p_i where that is zero throughout), and after the last
// accepted one another token from p_n: the tokens are then distributed as the target's.
//
// A draw is the inverse CDF: the smallest t with w_0 + ... + w_t > u (w_0 + ... + w_{V-1}).
// The weights are whole numbers, units of 2^-60 (a probability in [0, 2) rounded to the
// nearest, exact from 2^-37 on), so that sums are exact in any order: the token does not
// depend on how the vocabulary is shared out.
//
// A value becomes units by adding constants: x + 6 rounds x to a multiple of 2^-21 whose
// number is the sum's bits minus those of 6; what is left, exact, goes on with 1.5 * 2^-20
// (2^-43) and 1.5 * 2^-37 (2^-60).  Three integer sums then do for a row.  p and q take
// the two halves of packed instructions: about fifteen a pair of values, where shifts by
// the exponent take fifty and bound the large calls (256 sequences, 128000 tokens: 193 us,
// 84 without them).
//
// One cluster a sequence: every warp finds the row, sums its stretch of it in spans of 1 KB
// of p and of q, and sends the sum round; the CTA whose stretches hold the threshold goes on
// from the sums of a stretch's pieces, which its warps have kept, to the token.
//
// What bounds it: a small call its way through six dependent steps (bounds, drafted
// tokens, their probabilities, the row, the sums of all, the search: one sequence, 32000
// tokens, 5.3 us); a large one DRAM (256 sequences, 128000 tokens, up to 5 drafts, 190 MB:
// 44 us; 450 with 3, 400 MB: 64, 93 % of the copy rate), or, with bf16 rows, issue slots (72 %
// of them, for 15 instructions a token and what a span and a cluster cost: the same 256
// sequences, 95 MB: 36 us, 450 54).
//
// Spans come through a ring in shared memory, two ahead, in 16 bytes wherever p and q start.
// With loads of words into registers instead (six CTAs an SM, whose warps wait for their own
// loads) 450 sequences took 70 us, 300 without drafts 37 (33 now), the 256 in bf16 43, 248 of
// 150945 tokens in bf16 41 (35); with copies of words the 256 in fp32 57.  Four CTAs an SM
// with two spans ahead: two of three spans ahead 46, five with one 45 (and 450 without drafts
// 52, 47 now); spans of half the size 52 and more, of twice 46.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <type_traits>

#include "cluster.cuh"
#include "cluster_size.h"
#include "internal.h"
#include "tc_common.cuh"

namespace attn_skip {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int kMaxCluster = kLargeCluster;

template <bool BF16>
__device__ __forceinline__ uint32_t load_bits(const void *row, int64_t i) {  // as fp32 bits
  if constexpr (BF16) return (uint32_t)__ldg((const uint16_t *)row + i) << 16;
  else return __ldg((const uint32_t *)row + i);
}

constexpr float kM1 = 6.f;                   // 1.5 * 2^2: steps of 2^-21
constexpr float kM2 = 1.430511474609375e-6f; // 1.5 * 2^-20: steps of 2^-43
constexpr float kM3 = 1.0913936421275139e-11f; // 1.5 * 2^-37: steps of 2^-60
constexpr uint32_t kValid = 0x40000000u;     // fp32 bits from here on: 2 and more, NaN, negative

// Units of s1 steps of 2^-21, s2 of 2^-43 and s3 of 2^-60 (these two signed).
__device__ __forceinline__ u64 join(uint32_t s1, uint32_t s2, uint32_t s3) {
  return ((u64)s1 << 39) + ((u64)(int64_t)(int)s2 << 17) + (u64)(int64_t)(int)s3;
}

// A probability (fp32 bits) in units of 2^-60.  What lies outside [0, 2) (a NaN among it)
// counts as 0 and is noted; -0 is 0.
__device__ __forceinline__ u64 units(uint32_t b, bool &bad) {
  if (b >= kValid) {
    bad |= b != 0x80000000u;
    return 0;
  }
  const float x = __uint_as_float(b);
  const float t1 = x + kM1, r1 = x - (t1 - kM1);
  const float t2 = r1 + kM2, r2 = r1 - (t2 - kM2);
  const float t3 = r2 + kM3;
  return join(__float_as_uint(t1) - __float_as_uint(kM1),
              __float_as_uint(t2) - __float_as_uint(kM2), __float_as_uint(t3) - __float_as_uint(kM3));
}

struct Row {
  const void *p, *q;  // q null: only p counts
  int hole;           // a token whose weight is 0, or -1
};

template <bool BF16>
__device__ __forceinline__ u64 weight(const Row &r, int i, bool &bad) {
  const u64 p = units(load_bits<BF16>(r.p, i), bad);
  if (r.q) {
    const u64 q = units(load_bits<BF16>(r.q, i), bad);
    return p > q ? p - q : 0;
  }
  return i == r.hole ? 0 : p;
}

__device__ __forceinline__ u64 sum_warp(u64 x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ u64 scan_warp(u64 x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

// Rows that nobody has normalised may sum to 16 and more, past 64 bits: kTooMuch stands for
// their sum.  A second, coarse sum finds them out, since the two differ by 16 for every time that
// the first has wrapped.  A lane keeps it in steps of 2^-21, each value (or difference) to one
// step, and stops at kCoarse, 1024: a row's 2^22 values of a warp, the most that there are, and a
// token left out, leave it within a half of 16.  (One instruction a span.  By sums of 64 bits 450
// rows of 128000 in bf16 took 55.2 us, like this 54.2, without any 53.9; in fp32 65.2, 64.7 and
// 64.5; 300 without drafts 33.8, 33.8 and 33.0.)
constexpr u64 kTooMuch = ~0ull;
constexpr uint32_t kCoarse = 1u << 31;
__device__ __forceinline__ void add_coarse(uint32_t &sum, uint32_t x) {
  sum = __viaddmin_u32(sum, x, kCoarse);
}
__device__ __forceinline__ u64 unwrapped(u64 sum, uint32_t coarse) {
  const u64 all = ((u64)__reduce_add_sync(0xffffffffu, coarse >> 16) << 16) +
                  __reduce_add_sync(0xffffffffu, coarse & 0xffffu);
  return ((int64_t)all - (int64_t)(sum >> 39) + (1 << 24)) >> 25 > 0 ? kTooMuch : sum;
}

constexpr int kPieces = 64;  // sums of its stretch that a warp keeps, of a span each or several

// Two values' steps plus the constants' bits: a of the first, b of the second.
__device__ __forceinline__ void steps(uint32_t lo, uint32_t hi, uint32_t (&a)[3], uint32_t (&b)[3]) {
  auto two = [](float x, float y) {
    return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
  };
  const uint64_t m1 = two(kM1, kM1), m2 = two(kM2, kM2), m3 = two(kM3, kM3), neg = two(-1.f, -1.f);
  const uint64_t v = (uint64_t)lo | (uint64_t)hi << 32;
  const uint64_t t1 = tc::f2_add(v, m1);
  const uint64_t r1 = tc::f2_add(v, tc::f2_fma(t1, neg, m1));
  const uint64_t t2 = tc::f2_add(r1, m2);
  const uint64_t r2 = tc::f2_add(r1, tc::f2_fma(t2, neg, m2));
  const uint64_t t3 = tc::f2_add(r2, m3);
  a[0] = (uint32_t)t1; b[0] = (uint32_t)(t1 >> 32);
  a[1] = (uint32_t)t2; b[1] = (uint32_t)(t2 >> 32);
  a[2] = (uint32_t)t3; b[2] = (uint32_t)(t3 >> 32);
}

// A lane's sums.  Those of 512 values (16 a lane) fit in 32 bits: at most 2^22 steps of 2^-21
// each, none negative, and 2^21 of 2^-43, up or down; but a difference has up to 2^22 of those,
// so that half a warp's are summed before the others.
struct Sums {
  uint32_t s1 = 0, s2 = 0, s3 = 0;
  uint32_t most = 0;  // the largest bits of all values
  __device__ __forceinline__ void difference(uint32_t p, uint32_t q) {
    uint32_t a[3], b[3];
    most = max(most, max(p, q));
    steps(p, q, a, b);
    if (p > q) {  // (valid values: their bits compare as they do)
      s1 += a[0] - b[0];
      s2 += a[1] - b[1];
      s3 += a[2] - b[2];
    }
  }
  __device__ __forceinline__ void both(uint32_t p0, uint32_t p1) {
    uint32_t a[3], b[3];
    most = max(most, max(p0, p1));
    steps(p0, p1, a, b);
    s1 += a[0] + b[0] - 2 * __float_as_uint(kM1);
    s2 += a[1] + b[1] - 2 * __float_as_uint(kM2);
    s3 += a[2] + b[2] - 2 * __float_as_uint(kM3);
  }
  __device__ __forceinline__ u64 of_warp() const {
    return join(__reduce_add_sync(0xffffffffu, s1), __reduce_add_sync(0xffffffffu, s2),
                __reduce_add_sync(0xffffffffu, s3));
  }
};

// Slots are a row's tokens counted from the 16 bytes on in which p starts: token t of it is
// slot t + shift.  A warp takes spans of them, 1 KB of p and of q each, by asynchronous
// copies of 16 bytes ahead of the sums.  In shared memory slot i's q is `off` elements
// behind its p; words of two bf16 values come from two words where that is odd.
enum : int { kF32 = 0, kBf16 = 1, kBf16Across = 2 };
constexpr int U = 8;  // words of p, and of q, that a lane sums at a time
template <bool BF16> constexpr int kEach = BF16 ? 8 : 4;            // elements in 16 bytes
template <bool BF16> constexpr int kSpan = BF16 ? 64 * U : 32 * U;  // slots
constexpr int kStages = 3;             // spans that a warp has room for
constexpr int kSlot = 2 * 32 * U + 4;  // words of a span: 16 bytes more of q

__device__ __forceinline__ void copy_async(uint32_t smem, const void *gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

// Starts the copies for slots [i, min(i + kSpan, i1)).  Nothing is read from 16 bytes
// without a token of the row.
template <bool BF16, bool HAS_Q>
__device__ __forceinline__ void load_span(const Row &r, int i, int i1, int shift, int off, int lane,
                                          uint32_t *to) {
  constexpr int E = kEach<BF16>, SIZE = 16 / E;
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to) + lane * 16;
  // (16 bytes of p start where slot i does, those of q `off` elements before.)
  const uint8_t *p = (const uint8_t *)r.p + ((int64_t)(i - shift) * SIZE + lane * 16);
  const uint8_t *q = (const uint8_t *)r.q + ((int64_t)(i - shift - off) * SIZE + lane * 16);
  const int end = min(i + kSpan<BF16>, i1);
#pragma unroll
  for (int k = 0; k < U / 4; ++k) {
    const int t = i + (k * 32 + lane) * E;
    if (t < end) copy_async(at + k * 512, p + k * 512);
    if (HAS_Q && t - off < end && t - off + E > shift)
      copy_async(at + U * 128 + k * 512, q + k * 512);
  }
  if (HAS_Q && lane == 0 && i + kSpan<BF16> - off < end) copy_async(at + U * 256, q + U * 128);
}

// Sum of the weights of slots [i, min(i + kSpan, i1)), in every lane of the warp, out of `from`;
// a lane's `coarse` grows by the steps of its own.
template <int HOW, bool HAS_Q>
__device__ __forceinline__ u64 sum_span(const Row &r, int i, int i1, int shift, int off, int lane,
                                        uint32_t *from, uint32_t &coarse, bool &bad) {
  constexpr bool BF16 = HOW != kF32;
  Sums s;
  u64 sum = 0;
  if (i < shift || i + kSpan<BF16> > i1) {  // what is no token of the stretch counts as 0
    using Element = std::conditional_t<BF16, uint16_t, uint32_t>;
    Element *p = reinterpret_cast<Element *>(from);
    Element *q = reinterpret_cast<Element *>(from + U * 32) + off;
    if (lane < shift - i) p[lane] = q[lane] = 0;
#pragma unroll 1
    for (int t = i1 - i + lane; t < kSpan<BF16>; t += 32) p[t] = q[t] = 0;
    __syncwarp();
  }
  const uint32_t *x = from + lane, *y = x + U * 32 + (BF16 ? off >> 1 : off);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (BF16) {
      if (HAS_Q && u == U / 2) {
        sum = join(0, __reduce_add_sync(0xffffffffu, s.s2), 0);
        s.s2 = 0;
      }
      const uint32_t p = x[u * 32];
      if constexpr (HAS_Q) {
        uint32_t q = y[u * 32];
        if (HOW == kBf16Across) q = __byte_perm(q, y[u * 32 + 1], 0x5432);
        s.difference(p << 16, q << 16);
        s.difference(p & 0xffff0000u, q & 0xffff0000u);
      } else {
        s.both(p << 16, p & 0xffff0000u);
      }
    } else if constexpr (HAS_Q) {
      s.difference(x[u * 32], y[u * 32]);
    } else if (u % 2 == 0) {
      s.both(x[u * 32], x[u * 32 + 32]);
    }
  }
  if (__any_sync(0xffffffffu, s.most >= kValid)) {  // values to leave out: one by one
    u64 w = 0;
    uint32_t c = 0;
    for (int t = max(i, shift) + lane; t < min(i + kSpan<BF16>, i1); t += 32) {
      const u64 one = weight<BF16>(r, t - shift, bad);
      w += one;
      c += (uint32_t)(one >> 39);
    }
    add_coarse(coarse, c);
    return sum_warp(w);
  }
  add_coarse(coarse, s.s1);
  sum += s.of_warp();
  const int hole = r.hole + shift;
  if (r.hole < 0 || hole < i || hole >= min(i + kSpan<BF16>, i1)) return sum;
  bool noted = false;
  return sum - units(load_bits<BF16>(r.p, r.hole), noted);
}

// Sum of the weights of slots [i0, i1), in every lane, and of each `piece` of them (those mean
// nothing where the sum is kTooMuch).
template <int HOW, bool HAS_Q>
__device__ __forceinline__ u64 sum_stretch(const Row &r, int i0, int i1, int piece, u64 *pieces,
                                           int shift, int off, int lane, uint32_t *ring, bool &bad) {
  constexpr bool BF16 = HOW != kF32;
  constexpr int SPAN = kSpan<BF16>;
  auto load = [&](int i, int slot) {
    if (i < i1) load_span<BF16, HAS_Q>(r, i, i1, shift, off, lane, ring + slot * kSlot);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  u64 sum = 0;
  uint32_t coarse = 0;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) load(i0 + k * SPAN, k);
  int slot = 0;
  for (int i = i0, k = 0; i < i1; ++k) {
    u64 part = 0;
    for (const int end = min(i1, i + piece); i < end; i += SPAN) {
      __syncwarp();  // every lane is done with the span before, whose room is filled again
      load(i + (kStages - 1) * SPAN, slot == 0 ? kStages - 1 : slot - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // every lane's copies are there
      part += sum_span<HOW, HAS_Q>(r, i, i1, shift, off, lane, ring + slot * kSlot, coarse,
                                   bad);
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    if (lane == 0) pieces[k] = part;
    sum += part;
  }
  return unwrapped(sum, coarse);
}

template <bool BF16>
__global__ void __launch_bounds__(NT, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ u64 sums[2][kMaxCluster * NW];  // of every warp of the cluster
  __shared__ u64 pieces[NW][kPieces];        // of this CTA's stretches
  extern __shared__ __align__(16) uint32_t ring[];  // [NW][kStages][kSlot]
  const cg::cluster_group cluster = cg::this_cluster();
  cluster_started();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / n_cta;
  const int c0 = a.cu[s], c1 = a.cu[s + 1], n = c1 - c0;
  float us = a.u_sample[s];
  int32_t *out = a.tokens + (int64_t)s * (a.max_draft + 1);
  if (c0 < 0 || c1 < c0 || c1 > a.total || n > a.max_draft) {  // (the whole cluster)
    if (rank == 0) {
      for (int i = tid; i <= a.max_draft; i += NT) out[i] = -1;
      if (tid == 0) {
        a.n_accepted[s] = -1;
        atomicOr(a.err, kErrBadArg);
      }
    }
    cluster_wait();
    return;
  }
  const int esize = BF16 ? 2 : 4;
  auto target_row = [&](int i) {
    return (const uint8_t *)a.target + ((int64_t)c0 + s + i) * a.target_stride * esize;
  };
  auto draft_row = [&](int i) {
    return (const uint8_t *)a.draft + ((int64_t)c0 + i) * a.draft_stride * esize;
  };

  // The first rejected token: every warp for itself.
  bool bad = false;
  int acc = n, rejected = -1;  // accepted tokens; the rejected one
  for (int b = 0; b < n; b += 32) {
    const int i = b + lane;
    bool ok = true;
    int x = -1;
    if (i < n) {
      x = a.drafted[c0 + i];
      const float u = a.u_accept[c0 + i];
      const bool known = x >= 0 && x < a.V;
      bad |= !known || !(u >= 0.f && u < 1.f);
      ok = false;
      if (known) {
        const float p = __uint_as_float(load_bits<BF16>(target_row(i), x));
        const float q = a.draft ? __uint_as_float(load_bits<BF16>(draft_row(i), x)) : 1.f;
        ok = (double)u * (double)q < (double)p;  // (exact)
      }
    }
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    if (no) {
      acc = b + __ffs(no) - 1;
      rejected = __shfl_sync(0xffffffffu, x, acc - b);
      break;
    }
  }
  Row row{target_row(acc), nullptr, -1};
  if (acc < n) {
    if (a.draft) row.q = draft_row(acc);
    else row.hole = rejected;
  }

  cluster_wait();  // (the others' shared memory is there)
  const int all = n_cta * NW, mine = rank * NW + warp;
  auto behind = [](const void *row) {  // elements from the 16 bytes on that it starts in
    return (int)((uintptr_t)row / (16 / kEach<BF16>)) & (kEach<BF16> - 1);
  };
  const int shift = behind(row.p), off = (behind(row.q) - shift) & (kEach<BF16> - 1);
  const int slots = a.V + shift;
  // Every warp's stretch, a multiple of 64 slots, and the slots of which it keeps the sum.
  const int len = ((slots + all - 1) / all + 63) & ~63;
  const int i0 = min(mine * len, slots), i1 = min(i0 + len, slots);
  const int piece = (len + kPieces * kSpan<BF16> - 1) / (kPieces * kSpan<BF16>) * kSpan<BF16>;
  u64 total = 0, below = 0;  // sums of all warps, and of those of the CTAs before this one
  int round = 0;
  while (true) {  // a second time only where p - q is 0 throughout
    auto sum_as = [&](auto how, auto has_q) {
      return sum_stretch<how.value, has_q.value>(row, i0, i1, piece, pieces[warp], shift, off, lane,
                                                 ring + warp * (kStages * kSlot), bad);
    };
    using std::integral_constant;
    u64 stretch;
    if (!row.q) stretch = sum_as(integral_constant<int, BF16>{}, std::false_type{});
    else if (BF16 && (off & 1))
      stretch = sum_as(integral_constant<int, BF16 ? kBf16Across : kF32>{}, std::true_type{});
    else stretch = sum_as(integral_constant<int, BF16>{}, std::true_type{});
    if (lane < n_cta) *cluster.map_shared_rank(&sums[round][mine], lane) = stretch;
    cluster.sync();
    u64 before = 0, every = 0;
    uint32_t tops = 0;
    for (int i = lane; i < all; i += 32) {
      const u64 v = sums[round][i];
      every += v;
      tops += (uint32_t)(v >> 44);
      before += i < rank * NW ? v : 0;
    }
    total = sum_warp(every);
    // (Whether this sum has wrapped, by its terms' bits from 2^44 on.)
    tops = __reduce_add_sync(0xffffffffu, tops);
    if ((int)(tops - (uint32_t)(total >> 44) + (1u << 19)) >> 20 > 0) total = kTooMuch;
    below = sum_warp(before);
    if (round == 1 || total || acc == n) break;
    round = 1;
    row.q = nullptr;
    row.hole = -1;
  }
  if (!(us >= 0.f && us < 1.f)) {
    bad = true;
    us = us >= 1.f ? 0.99999994f : 0.f;
  }
  if (bad) atomicOr(a.err, kErrBadArg);
  const u64 threshold = __umul64hi(total, (u64)(us * 18446744073709551616.f));
  if (rank == 0)
    for (int i = tid; i <= a.max_draft; i += NT)
      if (i != acc) out[i] = i < acc ? a.drafted[c0 + i] : -1;
  if (rank == 0 && tid == 0) {
    a.n_accepted[s] = acc;
    if (!total || total == kTooMuch) out[acc] = a.V - 1;
  }
  if (total == kTooMuch) return;
  // The CTA whose stretches hold the threshold looks up the warp's, then the piece of it;
  // parts of that, where it is long, are summed again, until a load a thread is left.
  // `find`: which of n sums holds it; below becomes the sum before.
  auto find = [&](const u64 *part, int n) {
    for (int k = 0; k < n; k += 32) {
      const u64 v = k + lane < n ? part[k + lane] : 0, upto = below + scan_warp(v, lane);
      const unsigned here = __ballot_sync(0xffffffffu, threshold < upto && threshold >= upto - v);
      if (here) {
        below = __shfl_sync(0xffffffffu, upto - v, __ffs(here) - 1);
        return k + __ffs(here) - 1;
      }
      below = __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
  };
  // (The same for the whole CTA.)
  const int holder = find(&sums[round][rank * NW], NW);
  if (holder < 0) return;
  const int first = (rank * NW + holder) * len;
  const int k = find(pieces[holder], (min(len, slots - first) + piece - 1) / piece);
  if (k < 0) return;
  int lo = first + k * piece, end = min(min(lo + piece, first + len), slots);
  bool noted = false;
  auto weight_at = [&](int i) { return i < shift ? 0 : weight<BF16>(row, i - shift, noted); };
  while (end - lo > kSpan<BF16>) {
    const int step = ((end - lo + NW - 1) / NW + 31) & ~31;
    u64 sum = 0;
    const int last = min(lo + (warp + 1) * step, end);
#pragma unroll 4
    for (int i = lo + warp * step + lane; i < last; i += 32) sum += weight_at(i);
    sum = sum_warp(sum);
    __syncthreads();  // the sums before are no longer needed
    if (lane == 0) sums[0][warp] = sum;
    __syncthreads();
    const int part = find(sums[0], NW);
    if (part < 0) return;
    lo += part * step;
    end = min(lo + step, end);
  }
  constexpr int ONE = kSpan<BF16> / NT;
  const int j = lo + ONE * tid;
  const u64 w = j < end ? weight_at(j) : 0;
  const u64 all_w = w + (ONE == 2 && j + 1 < end ? weight_at(j + 1) : 0);
  const u64 of_warp = sum_warp(all_w);
  __syncthreads();
  if (lane == 0) sums[0][warp] = of_warp;
  __syncthreads();
  if (find(sums[0], NW) != warp) return;
  const u64 upto = below + scan_warp(all_w, lane);
  if (threshold < upto && threshold >= upto - all_w)
    out[acc] = (threshold < upto - all_w + w ? j : j + 1) - shift;
}

template <bool BF16>
cudaError_t launch(const VerifyArgs &a, int n_cta, cudaStream_t s) {
  constexpr int smem = NW * kStages * kSlot * (int)sizeof(uint32_t);
  const cudaError_t e = cudaFuncSetAttribute(verify_kernel<BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (n_cta == kLargeCluster && !large_cluster_fits((const void *)verify_kernel<BF16>, NT, smem))
    n_cta = kPortableCluster;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.n_seq * (unsigned)n_cta);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)n_cta;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<BF16>, a);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t s) {
  // CTAs a sequence: more while every warp has more than 256 tokens and
  //  - there are few (128000 tokens of one sequence: 38.8 us by one CTA, 8.4 by eight; 8000 of
  //    300: 8.2 by one, 18.7 by eight), or
  //  - all fit at once, four an SM, and each still has 16000 tokens (32000 of 210: 16.7 by one,
  //    14.2 by two; 50001 of 64: 10.7 by four, 11.3 by eight), or
  //  - each still has 60000 probabilities, so that they even out (128000 of 256, with drafts:
  //    47.2 by two, 44.1 by four, 46.7 by eight; of 300 without: 34.0 by one, 32.4 by two, 36.7
  //    by four; 32000 of 400, with drafts: 22.1 by one, 21.9 by two, 24.2 by four).
  // Sixteen where there are few and 3000 tokens for each (128000 tokens of one: 8.4 by eight,
  // 6.6 by sixteen; of 24: 11.2 and 10.3; 32000 of one in bf16: 5.7 and 6.2).
  // (Taken without the coarse sums, which add up to 2 % to all of them.)
  int n_cta = 1;
  while (n_cta < kMaxCluster && a.V > n_cta * NW * 256) {
    const int64_t ctas = (int64_t)n_cta * 2 * a.n_seq;
    const int each = a.V / (2 * n_cta);
    if (n_cta == 8 && (ctas > 400 || a.V < 48000)) break;
    if (ctas > 400 && (ctas > 608 || each < 16000) && each < (a.draft ? 30000 : 60000)) break;
    n_cta *= 2;
  }
  return a.bf16 ? launch<true>(a, n_cta, s) : launch<false>(a, n_cta, s);
}

}  // namespace attn_skip
