// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
// Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn_skip {

// Bits of the device error word.
enum : unsigned {
  kErrTimeout = 1u,  // a bounded mbarrier / flag wait gave up
  kErrBadArg = 2u,   // a device-side argument (a varlen length or threshold) was out of range
  kErrLayout = 4u,   // the dynamic shared-memory base was not 1024-byte aligned
};

struct PrefillArgs {
  const void *q, *k, *v;
  void *o;
  float *lse;
  uint32_t *bits;
  int B, Hq, Hkv, T, dk, dv, Br, Bc, causal;
  int n_t, n_b, words;  // tiles, blocks, bitmap words per tile
  float scale;          // natural-log scale applied to q.k
  float ln_lambda;      // -inf when lambda == 0
  unsigned *err;        // device error word
  // Statistics mode: margin [B,Hq,n_t,n_b] receives each traversed block's
  // statistic max_r(rowmax_r - m_new_r) (natural log; NaN = not traversed),
  // every block is treated as skipped, and o, lse, bits are not written.
  float *margin;
  int stats_only;
  // Explicit block set: [B,Hq,n_t,words] bit masks, bit j = block j is
  // traversed (within the causal range); null = every block.
  const uint32_t *block_set;
  // Variable-length batch: B sequences packed token-major, sequence b at
  // tokens [cu_seqlens[b], cu_seqlens[b+1]) of q [total,Hq,128], k and v
  // [total,Hkv,128] and o [total,Hq,128]; lse [Hq,total]; threshold
  // lambda_seq[b]; T = the longest length.  Null cu_seqlens = fixed length.
  const int32_t *cu_seqlens;
  const float *lambda_seq;
  int total;
};

struct DecodeArgs {
  const void *q, *k, *v;
  float *o_part, *lse_part;
  uint32_t *bits;
  int B, Hq, Hkv, L, dk, dv, Bc, n_splits;
  int64_t k_row_stride, v_row_stride;
  int n_b, bps, words;  // blocks, blocks per split (max), bitmap words per split
  float scale;
  float ln_lambda;
  unsigned *err;
  // Statistics mode: margin [B,Hkv,n_splits,bps] receives each block's
  // statistic over the query heads of the KV head (NaN past a split's last
  // block); every block is treated as skipped; o_part, lse_part, bits unused.
  float *margin;
  int stats_only;
  // Per-head decisions: bits [B,Hq,n_splits,words], each query head decides
  // for itself (the GQA kernel only).
  int per_head;
  // FP8 (E4M3) cache: k and v hold codes; one fp32 scale per (b, KV head)
  // for keys (multiplies the scores) and values (multiplies the outputs).
  const float *k_scale, *v_scale;
  // NVFP4 cache: k and v hold packed E2M1 codes [.., L, d/2], k_bs and v_bs
  // the E4M3 block scales [B,Hkv,L,d/16] (one per 16 elements of a row).
  const uint8_t *k_bs, *v_bs;
};

// Sampled decode output (SANTA estimator).
enum : int { kSantaIid = 0, kSantaSys = 1, kSantaStrat = 2 };

struct SantaArgs {
  const void *q, *k, *v;     // bf16 [B,Hq,128], [B,Hkv,L,128], [B,Hkv,L,128]
  const float *u;            // [B,Hq] (systematic) or [B,Hq,S] (stratified), in [0,1)
  float *scores;             // [B,Hq,n_b*128] stash: log2-scaled scores, -inf past L
  float *tile_stats;         // [B,Hq,n_tiles] (max, sum) pairs
  void *o;                   // [B,Hq,128] fp32 or bf16
  int32_t *idx;              // [B,Hq,S] sample indices, or null
  int B, Hq, Hkv, L, n_b, n_tiles, bps, S, mode, out_bf16;
  float scale;
  unsigned *err;
};

struct CombineArgs {
  const float *o_part, *lse_part;
  void *o;
  float *lse;
  int B, Hq, n_splits, dv;
  int out_bf16;
};

// The paged key/value cache (the fields of attn_kv_pages, checked).
enum : int { kKvBf16 = 0, kKvE4m3 = 1, kKvNvfp4 = 2 };

struct KvPages {
  int format, n_pages, page_size, Hkv;
  int page_shift;             // log2(page_size), -1 if it is no power of two
  int64_t page_stride;        // bytes from page to page in k and v
  void *k, *v;                // rows [n_pages][Hkv][page_size]
  uint8_t *k_scale, *v_scale; // E8M0 row scales [n_pages][Hkv][page_size]
  uint8_t *k_bs, *v_bs;       // NVFP4: E4M3 block scales [n_pages][Hkv][page_size][8]
};

struct KvAppendArgs {
  KvPages pages;
  const void *k_new, *v_new;           // [total][Hkv][128], tokens *_tok_stride elements apart
  int64_t k_tok_stride, v_tok_stride;
  int src_f32, n_seq, total, max_pages;
  const int32_t *cu_seqlens, *kv_len, *page_table;
  unsigned *err;
};

struct KvGatherArgs {
  KvPages pages;
  void *k_out, *v_out;                 // [total][Hkv][128]
  int out_f32, n_seq, total, max_pages;
  const int32_t *cu_rows, *start, *page_table;
  unsigned *err;
};

struct KvWidenArgs {
  KvPages pages;
  void *k_out, *v_out;                 // bf16 [n_seq][Hkv][stride][128]
  int n_seq, max_kv, stride, max_pages;
  const int32_t *kv_len, *page_table;
  unsigned *err;
};

// Attention of a chunk of new tokens per sequence over the paged cache.
struct ChunkArgs {
  KvPages pages;
  const void *q;                       // bf16 [total][Hq][128], tokens q_tok_stride elements apart
  int64_t q_tok_stride;
  void *o;                             // bf16 [total][Hq][128]
  float *lse;                          // [total][Hq]
  uint32_t *bits;                      // [n_seq][Hkv][n_t][n_splits][words], or null
  float *o_part, *lse_part;            // [total][Hq][n_splits][128] / [..][n_splits] (n_splits > 1)
  void *kv_work;                       // bf16 rows of a quantised cache, or null
  int n_seq, Hq, Hkv, G, TT;           // TT: tokens per tile, floor(128 / G)
  int total, max_chunk, max_kv, max_pages, causal;
  int n_splits, bps, n_t, words;       // bps: blocks per split
  const int32_t *cu_seqlens, *kv_len;
  const int32_t *page_table;           // null: sequence s's rows are page s
  const float *lambda;
  float scale;
  int shared_out;                      // decode: the CTAs share the batch out among themselves
  unsigned *err;
};

// Pages of several layers' caches (of one shape) in one launch.
constexpr int kMaxLayers = 64;

struct KvLayers {
  int n;
  int format, n_pages, page_size, Hkv, page_shift;
  int64_t page_stride;
  struct {
    uint8_t *k, *v, *k_scale, *v_scale, *k_bs, *v_bs;
  } layer[kMaxLayers];
};

struct CopyPagesArgs {
  KvLayers kv;
  int n_pairs;
  const int32_t *src, *dst;
  unsigned *err;
};

struct CompactArgs {
  KvLayers kv;
  int n_seq, total, max_pages, out_max_pages, per_head;
  const int32_t *cu_keep, *keep;       // keep [total], or [Hkv][total]
  const int32_t *start;                // [n_seq] or null
  const int32_t *table, *out_table;    // out_table null: in place
  int few, many;                       // in place: rows of the sequences of a launch
  unsigned *err;
};

struct ReserveArgs {
  int32_t *refs, *table;
  int n_pages, n_seq, max_pages, page_size;
  const int32_t *kv_len, *new_len;
  int32_t *got_len, *copy_src, *copy_dst;
  int rounds;                          // chunks of pages of a warp
  unsigned *err;
};

struct ForkArgs {
  int32_t *refs, *out_table;
  const int32_t *table, *kv_len, *new_len, *parent;  // parent null: rows stay in place
  int n_pages, n_seq, n_new, max_pages, page_size;
  unsigned *err;
};

// Drafted tokens against the target's probabilities.
struct VerifyArgs {
  const void *target, *draft;          // rows of V; draft null: each drafted token had q = 1
  int64_t target_stride, draft_stride; // elements
  int bf16, V, n_seq, total, max_draft;
  const int32_t *drafted, *cu;
  const float *u_accept, *u_sample;
  int32_t *tokens, *n_accepted;
  unsigned *err;
};

cudaError_t launch_kv_copy_pages(const CopyPagesArgs &a, cudaStream_t s);
cudaError_t launch_kv_compact(CompactArgs a, cudaStream_t s);
size_t pages_reserve_max_seqs();
size_t pages_reserve_max_pages();
cudaError_t launch_pages_reserve(ReserveArgs a, cudaStream_t s);
cudaError_t launch_pages_fork(const ForkArgs &a, cudaStream_t s);
cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t s);

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s);
cudaError_t launch_kv_widen(const KvWidenArgs &a, cudaStream_t s);
size_t chunk_paged_kv_bytes(int n_seq, int max_chunk, int max_kv, int Hkv, int TT, int format);
cudaError_t launch_kv_gather(const KvGatherArgs &a, cudaStream_t s);
cudaError_t launch_chunk_paged(const ChunkArgs &a, cudaStream_t s);
cudaError_t launch_decode_paged(const ChunkArgs &a, unsigned grid, cudaStream_t s);
int chunk_paged_splits(int n_seq, int total, int max_chunk, int max_kv, int Hkv, int TT, int format);

cudaError_t launch_prefill_f32(const PrefillArgs &a, cudaStream_t s);
cudaError_t launch_prefill_tc(const PrefillArgs &a, cudaStream_t s);
cudaError_t launch_decode_bf16(const DecodeArgs &a, cudaStream_t s);
cudaError_t launch_mla_decode(const DecodeArgs &a, cudaStream_t s);
cudaError_t launch_mla_cluster(const DecodeArgs &a, cudaStream_t s);
int mla_cluster_max_bps();
cudaError_t launch_decode_fp8(const DecodeArgs &a, cudaStream_t s);
cudaError_t launch_decode_nvfp4(const DecodeArgs &a, cudaStream_t s);
cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s);
cudaError_t launch_selftest_wait(unsigned *err, cudaStream_t s);
cudaError_t launch_santa_decode(const SantaArgs &a, cudaStream_t s);
size_t santa_sample_smem_bytes(int n_tiles, int S);

}  // namespace attn_skip
