// Host-side launchers of the library's kernels (one per .cu file), used by the
// C-ABI entry points.  Each returns the launch's cudaError_t.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// The driver's cuTensorMapEncodeTiled, looked up once through the runtime
// (nullptr if the driver does not provide it).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

cudaError_t launch_reshape_and_cache(const void* key, const void* value, void* cache,
                                     const int64_t* slot_mapping, int num_tokens,
                                     int num_kv_heads, int head_size, int block_size,
                                     int num_blocks, int* err, cudaStream_t stream);

// Offsets of a split-KV stage-1 launch that serves part of a larger
// computation (the suffix pass of cascade attention): every request skips its
// first seq_off tokens, whose blocks are the first table_col0 columns of its
// row, and split s writes slot ws_slot0 + s of a workspace with ws_slots
// slots per (request, head).
// logits (nullable): each token's logits as well, for the weights' sums.
struct DecodeExt {
  int table_col0;
  int seq_off;
  int ws_slots;
  int ws_slot0;
  float* logits = nullptr;   // [N, Hkv, logit_tokens, Hq / Hkv], log2 units
  int logit_tokens = 0;
};

// Split-KV stage 1; `chunk` = tokens per split (split_chunk in pa_common.cuh).
// ext == nullptr: no offsets, S slots.
cudaError_t launch_decode_splitkv(const void* q, const void* cache, const int32_t* block_table,
                                  const int32_t* seq_lens, int N, int Hq, int Hkv, int d, int bs,
                                  int num_blocks, int max_blocks, float scale, int S, int chunk,
                                  float* ws, int* err, cudaStream_t stream,
                                  const DecodeExt* ext = nullptr);

// MLA cache write: [kv_c | k_pe] rows of a [nb, bs, kv_lora_rank + rope_dim] pool.
cudaError_t launch_mla_cache_write(const void* kv_c, const void* k_pe, void* cache,
                                   const int64_t* slot_mapping, int num_tokens, int kv_lora_rank,
                                   int rope_dim, int block_size, int num_blocks, int* err,
                                   cudaStream_t stream);

// MLA prefill, step 1: expand every context token's latent through kv_b_proj
// into K_ws [N][s_max][H][192] = [k_nope | k_pe] and V_ws [N][s_max][H][128]
// (bf16).  Fixed widths: kv_lora_rank 512, rope 64, nope 128, v 128.
cudaError_t launch_mla_expand(const void* pool, const void* w_kv_b, const int32_t* block_table,
                              const int32_t* seq_lens, int N, int H, int bs, int num_blocks,
                              int max_blocks, int max_seq_len, int s_max, void* k_ws, void* v_ws,
                              int* err, cudaStream_t stream);

// fp8 (e4m3) pool: quantising cache write and split-KV stage 1.
cudaError_t launch_reshape_and_cache_fp8(const void* key, const void* value, void* cache,
                                         const int64_t* slot_mapping, int num_tokens,
                                         int num_kv_heads, int head_size, int block_size,
                                         int num_blocks, float k_scale, float v_scale, int* err,
                                         cudaStream_t stream);
cudaError_t launch_decode_splitkv_fp8(const void* q, const void* cache,
                                      const int32_t* block_table, const int32_t* seq_lens, int N,
                                      int Hq, int Hkv, int d, int bs, int num_blocks,
                                      int max_blocks, float scale, float k_scale, float v_scale,
                                      int S, int chunk, float* ws, int* err, cudaStream_t stream);

cudaError_t launch_lse_merge(const float* ws, int NH, int S, int dv, void* out, float* lse,
                             cudaStream_t stream);

// Varlen paged attention on tcgen05 tensor cores with TMA-gathered K/V.
struct VarlenLaunch {
  const void* q;
  const void* cache;
  const int32_t* block_table;
  const int32_t* qsl;
  const int32_t* seq_lens;
  int N, Hq, Hkv, d, bs, num_blocks, max_blocks, max_query_len;
  float scale;
  int causal;
  int window;              // > 0: sliding window of that many positions (causal)
  void* out;               // bf16 [T, Hq, d] (unused in partial mode)
  float* lse;              // [T, Hq], nullable (unused in partial mode)
  int* err;
  int table_col0 = 0;      // first table column of every request's row
  int seq_off = 0;         // tokens skipped at the front of every request
  int virt_total_q = 0;    // > 0: all rows [0, virt_total_q) as one request ...
  int virt_seq = 0;        // ... over virt_seq tokens of table row 0
  float* ws = nullptr;     // partial mode: fp32 [rows, Hq, ws_slots, d + 1]
  int ws_slots = 0;
  int ws_slot0 = 0;        // split s writes slot ws_slot0 + s
  int kv_splits = 1;
  int kv_chunk = 0;        // tokens per split, a multiple of 128
  // MLA prefill attention: keys [N * mla_s_max][Hkv][192] and values
  // [N * mla_s_max][Hkv][128] (the expanded workspaces) instead of the pool;
  // q is [T][Hkv][192], out [T][Hkv][128], one q head per kv head.
  const void* mla_k = nullptr;
  const void* mla_v = nullptr;
  int mla_s_max = 0;
};
cudaError_t launch_varlen_tc(const VarlenLaunch& L, cudaStream_t stream);

// Varlen attention with a causal sliding window and first tokens that stay
// visible (Hq / Hkv <= 128).
struct WindowPrefillLaunch {
  const void* q;
  const void* cache;
  const int32_t* block_table;
  const int32_t* qsl;
  const int32_t* seq_lens;
  int N, Hq, Hkv, d, bs, num_blocks, max_blocks, total_q, max_query_len;
  float scale;
  int window, sinks;
  void* out;    // bf16 [T, Hq, d]
  float* lse;   // [T, Hq], nullable
  int* err;
};
cudaError_t launch_window_prefill(const WindowPrefillLaunch& n, cudaStream_t stream);

// Causal attention over packed prompts (Hq / Hkv <= 128).
struct PromptLaunch {
  const void* q;
  const void* key;
  const void* value;
  int64_t q_stride, key_stride, value_stride;   // elements from token to token
  const int32_t* qsl;
  int N, Hq, Hkv, d, total_q, max_query_len;
  float scale;
  void* out;    // bf16 [T, Hq, d]
  float* lse;   // [T, Hq], nullable
  int* err;
};
cudaError_t launch_prompt(const PromptLaunch& n, cudaStream_t stream);

// Decode with a sliding window and first tokens that stay visible, bf16 or
// e4m3 pool, in one launch.
struct DecodeWindowLaunch {
  const void* q;
  const void* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int N, Hq, Hkv, d, bs, num_blocks, max_blocks, window, sinks;
  float scale, k_scale, v_scale;   // k_scale, v_scale 1 for bf16
  bool fp8;
  void* out;
  float* lse;
  int* err;
  int sm_count;
};
cudaError_t launch_decode_window(const DecodeWindowLaunch& n, cudaStream_t stream);

// 4-bit pool: quantising cache write, and decode with or without the weights' sums.
cudaError_t launch_cache_write_fp4(const void* key, const void* value, int64_t key_stride,
                                   int64_t value_stride, void* cache, const int64_t* slot_mapping,
                                   int num_tokens, int num_kv_heads, int head_size, int block_size,
                                   int num_blocks, float k_scale, float v_scale, int* err,
                                   cudaStream_t stream);
struct DecodeFp4Launch {
  const void* q;
  const void* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int N, Hq, Hkv, d, bs, num_blocks, max_blocks;
  float scale, k_scale, v_scale;
  int max_seq_len;
  void* workspace;    // decode_fp4_workspace's bytes
  float* scores;      // [N, Hkv, score_tokens], or null: no sums
  int score_tokens;
  void* out;
  float* lse;
  int* err;
  int sm_count;
};
cudaError_t launch_decode_fp4(const DecodeFp4Launch& n, cudaStream_t stream);
// Offsets in the workspace, and its size.
struct Fp4Workspace {
  size_t held, cut, parts, spans, row_lse, logits, bytes;
};
Fp4Workspace decode_fp4_workspace(int N, int Hq, int Hkv, int d, int max_seq_len, bool sums,
                                  int sm_count);

// Merge of what stage 1 left, and each token's weights (exp2 of its logit less the
// row's log-sum-exp, summed over the group's heads) added to scores [N, Hkv,
// score_tokens].  Stage 1 left either S partials of each row (ws), or outputs and
// log-sum-exps of the units that were not cut and states of those that were (spans).
struct ScoresLaunch {
  const float* ws;        // [N, Hq, S, d + 1], or null:
  int S;
  const float* parts;     // [CTA][2][Hq / Hkv][d + 2]
  const int2* spans;      // [N, Hkv] first and last CTA
  const float* row_lse;   // [N, Hq]
  float out_scale;
  const float* logits;
  int logit_tokens;
  const int32_t* seq_lens;
  int positions;          // with spans: of a table row
  int N, Hq, Hkv, d, max_seq_len;
  float* scores;
  int score_tokens;
  void* out;
  float* lse;
  int* err;
};
cudaError_t launch_decode_scores(const ScoresLaunch& n, cudaStream_t stream);

// Eviction by accumulated weights, and the lengths and blocks behind it.
struct EvictLaunch {
  void* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* scores;
  float* new_scores;      // may be scores
  int32_t* new_lens;      // may be seq_lens
  int32_t* kept;          // [N, Hkv, budget]
  int32_t* free_blocks;   // nullable
  const int32_t* free_start;
  int32_t* new_free_start;
  int num_free;
  int N, Hkv, d, bs, num_blocks, max_blocks, score_tokens, budget, recent, first;
  bool four;              // 4-bit pool; else rows of row_bytes in the standard layout
  int row_bytes;
  int* err;
};
cudaError_t launch_evict(const EvictLaunch& n, cudaStream_t stream);

// Step plan: query_start_loc, seq_lens, positions, slot_mapping and new table
// entries from the requests' lengths.
cudaError_t launch_plan_step(const int32_t* context_lens, const int32_t* query_lens,
                             const int32_t* free_blocks, const int32_t* free_start, int num_free,
                             int num_seqs, int max_blocks, int bs, int num_blocks, int max_tokens,
                             int32_t* block_table, int32_t* query_start_loc, int32_t* seq_lens,
                             int32_t* positions, int64_t* slot_mapping, int32_t* totals, int* err,
                             cudaStream_t stream);

// Head norms, rotation and cache write in one pass (bf16 or e4m3 pool).
struct NormRopeLaunch {
  const void* q;
  const void* key;
  const void* value;
  int64_t q_stride, key_stride, value_stride;   // elements from token to token
  const void* q_weight;                         // both or neither
  const void* k_weight;
  float eps;
  const float* cos_sin;
  int max_position, rotary_dim, interleaved;
  const int32_t* positions;
  void* cache;
  const int64_t* slot_mapping;
  int num_tokens, Hq, Hkv, d, bs, num_blocks;
  bool fp8;
  float k_scale, v_scale;
  void* q_out;
  int* err;
  int sm_count;
};
cudaError_t launch_norm_rope(const NormRopeLaunch& n, cudaStream_t stream);

// MLA stage 1 on tcgen05 tensor cores + merge.
cudaError_t launch_mla_tc(const void* q, const void* cache, const int32_t* block_table,
                          const int32_t* seq_lens, int B, int H, int bs, int num_blocks,
                          int max_blocks, float scale, int S, int chunk, float* ws, void* out,
                          float* lse, int* err, cudaStream_t stream);

// Device address of the error word on the current device (nullptr on error).
int* device_error_word();

}  // namespace pa
