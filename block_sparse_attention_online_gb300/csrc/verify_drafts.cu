// Drafted tokens against the target's probabilities (speculative sampling).
//
// Drafted token i of a sequence, drawn from q_i, is accepted if u_i q_i(x_i) < p_i(x_i)
// and all before it are; at the first rejected one the token is drawn from the positive
// part of p_i - q_i instead (from p_i where that is zero throughout), and after the last
// accepted one another token from p_n: the tokens are then distributed as the target's.
//
// A draw is the inverse CDF: the smallest t with w_0 + ... + w_t > u (w_0 + ... + w_{V-1}).
// The weights are whole numbers, units of 2^-60 (a probability in [0, 2) truncated to that,
// exact from 2^-37 on), so that sums are exact in any order: the token does not depend on
// how the vocabulary is shared out.
//
// One cluster a sequence: every CTA finds the row, sums its warps' stretches of it, and
// sends the sums round; the warp whose stretch holds the threshold finds the token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"

namespace attn_skip {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int NT = 512;
constexpr int NW = NT / 32;
constexpr int kMaxCluster = 16;

template <bool BF16>
__device__ __forceinline__ uint32_t load_bits(const void *row, int64_t i) {  // as fp32 bits
  if constexpr (BF16) return (uint32_t)__ldg((const uint16_t *)row + i) << 16;
  else return __ldg((const uint32_t *)row + i);
}

// A probability (fp32 bits) in units of 2^-60, truncated.  What lies outside [0, 2) (a NaN
// among it) counts as 0 and is noted; -0 is 0.
__device__ __forceinline__ u64 units(uint32_t b, bool &bad) {
  const int e = (int)(b >> 23);
  const uint32_t m = (b & 0x7fffffu) | 0x800000u;
  if (b >= 0x40000000u) {
    bad |= b != 0x80000000u;
    return 0;
  }
  // b = m 2^(e - 150) = m 2^(e - 90) units; subnormals (e = 0) vanish.
  const int sh = e - 90;
  return sh >= 0 ? (u64)m << sh : sh > -24 ? (u64)(m >> -sh) : 0;
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

template <bool BF16>
__global__ void __launch_bounds__(NT) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ u64 sums[2][kMaxCluster * NW];  // of every warp of the cluster
  __shared__ int first_rejected;
  const cg::cluster_group cluster = cg::this_cluster();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / n_cta;
  const int c0 = a.cu[s], c1 = a.cu[s + 1], n = c1 - c0;
  int32_t *out = a.tokens + (int64_t)s * (a.max_draft + 1);
  if (c0 < 0 || c1 < c0 || c1 > a.total || n > a.max_draft) {  // (the whole cluster)
    if (rank == 0) {
      for (int i = tid; i <= a.max_draft; i += NT) out[i] = -1;
      if (tid == 0) {
        a.n_accepted[s] = -1;
        atomicOr(a.err, kErrBadArg);
      }
    }
    return;
  }
  const int esize = BF16 ? 2 : 4;
  auto target_row = [&](int i) {
    return (const uint8_t *)a.target + ((int64_t)c0 + s + i) * a.target_stride * esize;
  };
  auto draft_row = [&](int i) {
    return (const uint8_t *)a.draft + ((int64_t)c0 + i) * a.draft_stride * esize;
  };

  // The first rejected token.
  bool bad = false;
  if (tid == 0) first_rejected = n;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const int x = a.drafted[c0 + i];
    const float u = a.u_accept[c0 + i];
    bool ok = false;
    if (x < 0 || x >= a.V || !(u >= 0.f && u < 1.f)) {
      bad = true;
    }
    if (x >= 0 && x < a.V) {
      const float p = __uint_as_float(load_bits<BF16>(target_row(i), x));
      const float q = a.draft ? __uint_as_float(load_bits<BF16>(draft_row(i), x)) : 1.f;
      ok = (double)u * (double)q < (double)p;  // (exact)
    }
    if (!ok) atomicMin(&first_rejected, i);
  }
  __syncthreads();
  const int acc = first_rejected;
  Row row{target_row(acc), nullptr, -1};
  if (acc < n) {
    if (a.draft) row.q = draft_row(acc);
    else row.hole = a.drafted[c0 + acc];
  }

  // Every warp's stretch, a multiple of 32 tokens.
  const int all = n_cta * NW, mine = rank * NW + warp;
  const int len = ((a.V + all - 1) / all + 31) & ~31;
  const int i0 = (int)min((int64_t)mine * len, (int64_t)a.V), i1 = min(i0 + len, a.V);
  u64 total = 0, before = 0, stretch = 0;
  for (int round = 0; round < 2; ++round) {  // the second one only where p - q is 0 throughout
    u64 w = 0;
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) w += weight<BF16>(row, i, bad);
    w = sum_warp(w);
    if (lane < n_cta) *cluster.map_shared_rank(&sums[round][mine], lane) = w;
    cluster.sync();
    // Sums of all warps, and of those before this one.
    u64 below = 0, every = 0;
    for (int i = lane; i < all; i += 32) {
      const u64 v = sums[round][i];
      every += v;
      below += i < mine ? v : 0;
    }
    total = sum_warp(every);
    before = sum_warp(below);
    stretch = w;
    if (total || acc == n) break;
    row.q = nullptr;
    row.hole = -1;
  }
  if (bad) atomicOr(a.err, kErrBadArg);

  float u = a.u_sample[s];
  if (!(u >= 0.f && u < 1.f)) {
    if (rank == 0 && tid == 0) atomicOr(a.err, kErrBadArg);
    u = u >= 1.f ? 0.99999994f : 0.f;
  }
  const u64 threshold = __umul64hi(total, (u64)(u * 18446744073709551616.f));
  if (rank == 0)
    for (int i = tid; i <= a.max_draft; i += NT)
      if (i != acc) out[i] = i < acc ? a.drafted[c0 + i] : -1;
  if (rank == 0 && tid == 0) {
    a.n_accepted[s] = acc;
    if (!total) out[acc] = a.V - 1;
  }
  if (threshold < before || threshold - before >= stretch) return;
  // The stretch that holds the threshold: a piece a lane, then the lane's piece.
  const int piece = len / 32, j0 = min(i0 + lane * piece, i1), j1 = min(j0 + piece, i1);
  u64 w = 0;
  bool noted = false;
  for (int i = j0; i < j1; ++i) w += weight<BF16>(row, i, noted);
  const u64 upto = before + scan_warp(w, lane);
  if (threshold < upto && threshold >= upto - w) {
    u64 f = upto - w;
    for (int i = j0; i < j1; ++i) {
      f += weight<BF16>(row, i, noted);
      if (f > threshold) {
        out[acc] = i;
        break;
      }
    }
  }
}

template <bool BF16>
cudaError_t launch(const VerifyArgs &a, int n_cta, cudaStream_t s) {
  if (n_cta > 8) {
    const cudaError_t e = cudaFuncSetAttribute(
        verify_kernel<BF16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.n_seq * (unsigned)n_cta);
  cfg.blockDim = dim3(NT);
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
  // CTAs a sequence: as many as leave every warp 128 tokens, up to eight.
  int n_cta = 1;
  while (n_cta < 8 && (int64_t)n_cta * NW * 128 < a.V) n_cta *= 2;
  return a.bf16 ? launch<true>(a, n_cta, s) : launch<false>(a, n_cta, s);
}

}  // namespace attn_skip
