// C-ABI entry points of libpa.so (declared in include/pa.h): host-side
// validation, split planning and kernel launches.  Nothing here allocates
// device memory or synchronises the host (except pa_get_device_error, which
// is a diagnostic).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

// The device error word (PA_DEVERR_* bits).  Kernels receive its address.
__device__ int g_device_error = 0;

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace pa

namespace {

constexpr int kMaxSplits = 16384;   // the merge keeps S weights in shared memory
constexpr int kMaxGridYZ = 65535;

bool shape_ok(const pa_shape* s) {
  return s != nullptr && s->num_seqs >= 0 && s->num_q_heads > 0 && s->num_kv_heads > 0 &&
         s->head_size > 0 && s->block_size > 0 && s->num_blocks > 0 &&
         s->max_blocks_per_seq > 0 && s->num_q_heads % s->num_kv_heads == 0 &&
         s->block_size % 16 == 0 && s->num_seqs <= kMaxGridYZ && s->num_kv_heads <= kMaxGridYZ;
}

pa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// The kernels move cache rows and MLA queries in 16-byte vectors and q / out
// rows in 4-byte pairs.
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

bool scale_ok(float x) { return x > 0.f && x <= 3.4028234663852886e38f; }

// The windowed kernels multiply logits by scale * k_scale * log2(e) in fp32, which
// has to stay finite (0 * inf is NaN).
bool logit_scale_ok(float scale, float k_scale) {
  return scale_ok(scale) && scale_ok(k_scale) &&
         scale * k_scale * pa::kLog2e <= 3.4028234663852886e38f;
}

// A range of device memory.
struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

// Device address of the error word on the current device (looked up once per
// device; a host-side symbol is not a device address).
int* device_error_ptr() {
  static std::mutex mu;
  static int* cached[64] = {nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && cached[dev] != nullptr) return cached[dev];
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, pa::g_device_error) != cudaSuccess) return nullptr;
  if (dev < 64) cached[dev] = static_cast<int*>(p);
  return static_cast<int*>(p);
}

}  // namespace

namespace pa {
// The error word's device address for kernels launched from other files.
int* device_error_word() { return device_error_ptr(); }
}  // namespace pa

namespace {

pa::VarlenLaunch varlen_launch(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* qsl, const int32_t* seq_lens, int max_query_len,
                               const pa_shape* shape, float scale, int causal, int window,
                               void* out, float* lse) {
  pa::VarlenLaunch L{};
  L.q = q;
  L.cache = kv_cache;
  L.block_table = block_table;
  L.qsl = qsl;
  L.seq_lens = seq_lens;
  L.N = shape->num_seqs;
  L.Hq = shape->num_q_heads;
  L.Hkv = shape->num_kv_heads;
  L.d = shape->head_size;
  L.bs = shape->block_size;
  L.num_blocks = shape->num_blocks;
  L.max_blocks = shape->max_blocks_per_seq;
  L.max_query_len = max_query_len;
  L.scale = scale;
  L.causal = causal;
  L.window = window;
  L.out = out;
  L.lse = lse;
  L.err = device_error_ptr();
  return L;
}

}  // namespace

extern "C" {

pa_status pa_reshape_and_cache(const void* key, const void* value, void* kv_cache,
                               const int64_t* slot_mapping, int num_tokens,
                               const pa_shape* shape, void* stream) {
  if (shape == nullptr || num_tokens < 0) return PA_ERR_INVALID;
  if (shape->num_kv_heads <= 0 || shape->head_size <= 0 || shape->block_size <= 0 ||
      shape->block_size % 16 != 0 || shape->num_blocks <= 0)
    return PA_ERR_INVALID;
  if (shape->head_size % 8 != 0) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (key == nullptr || value == nullptr || kv_cache == nullptr || slot_mapping == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_reshape_and_cache(key, value, kv_cache, slot_mapping, num_tokens,
                                                shape->num_kv_heads, shape->head_size,
                                                shape->block_size, shape->num_blocks,
                                                device_error_ptr(),
                                                static_cast<cudaStream_t>(stream)));
}

pa_status pa_mla_cache_write(const void* kv_c, const void* k_pe, void* kv_cache,
                             const int64_t* slot_mapping, int num_tokens, int kv_lora_rank,
                             int rope_dim, int block_size, int num_blocks, void* stream) {
  if (num_tokens < 0 || kv_lora_rank <= 0 || rope_dim < 0 || block_size <= 0 ||
      block_size % 16 != 0 || num_blocks <= 0)
    return PA_ERR_INVALID;
  if (kv_lora_rank % 8 != 0 || rope_dim % 8 != 0) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (kv_c == nullptr || (k_pe == nullptr && rope_dim > 0) || kv_cache == nullptr ||
      slot_mapping == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(kv_c, 16) || !aligned(k_pe, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_mla_cache_write(kv_c, k_pe, kv_cache, slot_mapping, num_tokens,
                                              kv_lora_rank, rope_dim, block_size, num_blocks,
                                              device_error_ptr(),
                                              static_cast<cudaStream_t>(stream)));
}

size_t pa_mla_prefill_workspace_bytes(int num_seqs, int max_seq_len, int num_heads) {
  if (num_seqs < 0 || max_seq_len < 0 || num_heads <= 0) return 0;
  return static_cast<size_t>(num_seqs) * max_seq_len * num_heads * (192 + 128) * 2;
}

static bool mla_prefill_shape_ok(int num_seqs, int num_heads, int block_size, int num_blocks,
                                 int max_blocks_per_seq, int max_seq_len) {
  return num_seqs >= 0 && num_seqs <= kMaxGridYZ && num_heads > 0 && num_heads <= kMaxGridYZ &&
         block_size > 0 && block_size % 16 == 0 && num_blocks > 0 && max_blocks_per_seq > 0 &&
         max_seq_len >= 0;
}

pa_status pa_mla_expand_kv(const void* kv_cache, const void* w_kv_b, const int32_t* block_table,
                           const int32_t* seq_lens, int num_seqs, int num_heads, int block_size,
                           int num_blocks, int max_blocks_per_seq, int max_seq_len, void* k_ws,
                           void* v_ws, void* stream) {
  if (!mla_prefill_shape_ok(num_seqs, num_heads, block_size, num_blocks, max_blocks_per_seq,
                            max_seq_len))
    return PA_ERR_INVALID;
  if (num_seqs == 0 || max_seq_len == 0) return PA_OK;
  if (kv_cache == nullptr || w_kv_b == nullptr || block_table == nullptr ||
      seq_lens == nullptr || k_ws == nullptr || v_ws == nullptr)
    return PA_ERR_INVALID;
  // The expansion writes its rows with 32-byte stores.
  if (!aligned(kv_cache, 16) || !aligned(w_kv_b, 16) || !aligned(k_ws, 32) || !aligned(v_ws, 32))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_mla_expand(kv_cache, w_kv_b, block_table, seq_lens, num_seqs,
                                         num_heads, block_size, num_blocks, max_blocks_per_seq,
                                         max_seq_len, max_seq_len, k_ws, v_ws,
                                         device_error_ptr(), static_cast<cudaStream_t>(stream)));
}

pa_status pa_mla_prefill(const void* q, const void* kv_cache, const void* w_kv_b,
                         const int32_t* block_table, const int32_t* query_start_loc,
                         const int32_t* seq_lens, int total_q, int max_query_len, int num_seqs,
                         int num_heads, int block_size, int num_blocks, int max_blocks_per_seq,
                         int max_seq_len, float scale, int causal, void* workspace, void* out,
                         float* lse, void* stream) {
  if (!mla_prefill_shape_ok(num_seqs, num_heads, block_size, num_blocks, max_blocks_per_seq,
                            max_seq_len) ||
      total_q < 0 || max_query_len < 0)
    return PA_ERR_INVALID;
  if (total_q == 0 || num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || w_kv_b == nullptr || block_table == nullptr ||
      query_start_loc == nullptr || seq_lens == nullptr || workspace == nullptr || out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(w_kv_b, 16) ||
      !aligned(workspace, 32) || !aligned(out, 16) || !aligned(lse, 4))
    return PA_ERR_INVALID;
  const long long rows = static_cast<long long>(num_seqs) * max_seq_len;
  if (rows * num_heads > INT_MAX) return PA_ERR_INVALID;   // 3-D map row coordinate
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* k_ws = static_cast<uint8_t*>(workspace);
  uint8_t* v_ws = k_ws + rows * num_heads * 192 * 2;
  if (pa::launch_mla_expand(kv_cache, w_kv_b, block_table, seq_lens, num_seqs, num_heads,
                            block_size, num_blocks, max_blocks_per_seq, max_seq_len, max_seq_len,
                            k_ws, v_ws, device_error_ptr(), st) != cudaSuccess)
    return PA_ERR_CUDA;
  pa::VarlenLaunch L{};
  L.q = q;
  L.cache = kv_cache;
  L.block_table = block_table;
  L.qsl = query_start_loc;
  L.seq_lens = seq_lens;
  L.N = num_seqs;
  L.Hq = num_heads;
  L.Hkv = num_heads;
  L.d = 192;
  L.bs = block_size;
  L.num_blocks = num_blocks;
  L.max_blocks = max_blocks_per_seq;
  L.max_query_len = max_query_len;
  L.scale = scale;
  L.causal = causal ? 1 : 0;
  L.window = 0;
  L.out = out;
  L.lse = lse;
  L.err = device_error_ptr();
  L.mla_k = k_ws;
  L.mla_v = v_ws;
  L.mla_s_max = max_seq_len;
  return from_cuda(pa::launch_varlen_tc(L, st));
}

pa_status pa_varlen_fwd(const void* q, const void* kv_cache, const int32_t* block_table,
                        const int32_t* query_start_loc, const int32_t* seq_lens, int total_q,
                        int max_query_len, const pa_shape* shape, float scale, int causal,
                        void* out, float* lse, void* stream) {
  if (!shape_ok(shape) || total_q < 0 || max_query_len < 0) return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (total_q == 0 || shape->num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr ||
      query_start_loc == nullptr || seq_lens == nullptr || out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_varlen_tc(
      varlen_launch(q, kv_cache, block_table, query_start_loc, seq_lens, max_query_len, shape,
                    scale, causal ? 1 : 0, 0, out, lse),
      static_cast<cudaStream_t>(stream)));
}

pa_status pa_varlen_fwd_window(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* query_start_loc, const int32_t* seq_lens,
                               int total_q, int max_query_len, const pa_shape* shape, float scale,
                               int sliding_window, void* out, float* lse, void* stream) {
  if (!shape_ok(shape) || total_q < 0 || max_query_len < 0 || sliding_window < 1)
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (total_q == 0 || shape->num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr ||
      query_start_loc == nullptr || seq_lens == nullptr || out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_varlen_tc(
      varlen_launch(q, kv_cache, block_table, query_start_loc, seq_lens, max_query_len, shape,
                    scale, 1, sliding_window, out, lse),
      static_cast<cudaStream_t>(stream)));
}

pa_status pa_varlen_fwd_sinks(const void* q, const void* kv_cache, const int32_t* block_table,
                              const int32_t* query_start_loc, const int32_t* seq_lens,
                              int total_q, int max_query_len, const pa_shape* shape, float scale,
                              int sliding_window, int num_sinks, void* out, float* lse,
                              void* stream) {
  if (!shape_ok(shape) || total_q < 0 || max_query_len < 0 || sliding_window < 1 ||
      num_sinks < 0 || !logit_scale_ok(scale, 1.f))
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 128) return PA_ERR_UNSUPPORTED;
  if (total_q == 0 || shape->num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr ||
      query_start_loc == nullptr || seq_lens == nullptr || out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(query_start_loc, 4) || !aligned(seq_lens, 4))
    return PA_ERR_INVALID;
  pa::WindowPrefillLaunch n{};
  n.q = q;
  n.cache = kv_cache;
  n.block_table = block_table;
  n.qsl = query_start_loc;
  n.seq_lens = seq_lens;
  n.N = shape->num_seqs;
  n.Hq = shape->num_q_heads;
  n.Hkv = shape->num_kv_heads;
  n.d = shape->head_size;
  n.bs = shape->block_size;
  n.num_blocks = shape->num_blocks;
  n.max_blocks = shape->max_blocks_per_seq;
  n.total_q = total_q;
  n.max_query_len = max_query_len;
  n.scale = scale;
  n.window = sliding_window;
  n.sinks = num_sinks;
  n.out = out;
  n.lse = lse;
  n.err = device_error_ptr();
  return from_cuda(pa::launch_window_prefill(n, static_cast<cudaStream_t>(stream)));
}

pa_status pa_prompt_fwd(const void* q, const void* key, const void* value, int64_t q_stride,
                        int64_t key_stride, int64_t value_stride, const int32_t* query_start_loc,
                        int num_seqs, int total_q, int max_query_len, int num_q_heads,
                        int num_kv_heads, int head_size, float scale, void* out, float* lse,
                        void* stream) {
  if (num_seqs < 0 || num_seqs > kMaxGridYZ || total_q < 0 || max_query_len < 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > kMaxGridYZ || head_size <= 0 ||
      num_q_heads % num_kv_heads != 0 || !logit_scale_ok(scale, 1.f))
    return PA_ERR_INVALID;
  if ((head_size != 64 && head_size != 128) || num_q_heads / num_kv_heads > 128)
    return PA_ERR_UNSUPPORTED;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_size;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_size;
  // (A tensor map's strides are below 2^40 bytes.)
  constexpr int64_t kMost = 1LL << 38;
  if (q_stride < qw || key_stride < kw || value_stride < kw || q_stride % 8 != 0 ||
      key_stride % 8 != 0 || value_stride % 8 != 0 || q_stride > kMost || key_stride > kMost ||
      value_stride > kMost)
    return PA_ERR_INVALID;
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || key == nullptr || value == nullptr || query_start_loc == nullptr ||
      out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(query_start_loc, 4))
    return PA_ERR_INVALID;
  auto rows = [&](const void* p, int64_t stride, int64_t width) {
    return Range{p, static_cast<size_t>((total_q - 1) * stride + width) * 2};   // bf16
  };
  const Range o = rows(out, qw, qw);
  if (overlap(o, rows(q, q_stride, qw)) || overlap(o, rows(key, key_stride, kw)) ||
      overlap(o, rows(value, value_stride, kw)))
    return PA_ERR_INVALID;
  pa::PromptLaunch n{};
  n.q = q;
  n.key = key;
  n.value = value;
  n.q_stride = q_stride;
  n.key_stride = key_stride;
  n.value_stride = value_stride;
  n.qsl = query_start_loc;
  n.N = num_seqs;
  n.Hq = num_q_heads;
  n.Hkv = num_kv_heads;
  n.d = head_size;
  n.total_q = total_q;
  n.max_query_len = max_query_len;
  n.scale = scale;
  n.out = out;
  n.lse = lse;
  n.err = device_error_ptr();
  return from_cuda(pa::launch_prompt(n, static_cast<cudaStream_t>(stream)));
}

int pa_cascade_prefix_splits(int total_q, int num_q_heads, int num_kv_heads,
                             int prefix_tokens, int sm_count) {
  if (total_q <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || prefix_tokens <= 0) return 1;
  if (sm_count <= 0) sm_count = pa_device_sm_count();
  if (sm_count <= 0) sm_count = 1;
  // One CTA per (256 packed rows, kv head, split) and one CTA per SM: split
  // the prefix until every SM has a unit, at most one split per 128 tokens.
  const long long rows = static_cast<long long>(total_q) * (num_q_heads / num_kv_heads);
  const long long units = ((rows + 255) / 256) * num_kv_heads;
  long long s = (sm_count + units - 1) / units;
  const long long by_len = (static_cast<long long>(prefix_tokens) + 127) / 128;
  if (s > by_len) s = by_len;
  if (s > kMaxSplits - 1) s = kMaxSplits - 1;
  return s < 1 ? 1 : static_cast<int>(s);
}

pa_status pa_cascade_fwd(const void* q, const void* kv_cache, const int32_t* block_table,
                         const int32_t* query_start_loc, const int32_t* seq_lens, int total_q,
                         int max_query_len, int max_seq_len, int num_common_prefix_blocks,
                         int num_prefix_splits, int num_suffix_splits, const pa_shape* shape,
                         float scale, int causal, float* workspace, void* out, float* lse,
                         void* stream) {
  if (!shape_ok(shape) || total_q < 0 || max_query_len < 0 || max_seq_len < 0 ||
      num_common_prefix_blocks < 0 || num_common_prefix_blocks > shape->max_blocks_per_seq ||
      num_prefix_splits < 1 || num_suffix_splits < 1 ||
      num_prefix_splits + num_suffix_splits > kMaxSplits)
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 16) return PA_ERR_UNSUPPORTED;
  if (total_q == 0 || shape->num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr ||
      query_start_loc == nullptr || seq_lens == nullptr || out == nullptr || workspace == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 4))
    return PA_ERR_INVALID;
  const long long prefix_tokens =
      static_cast<long long>(num_common_prefix_blocks) * shape->block_size;
  const long long nh = static_cast<long long>(total_q) * shape->num_q_heads;
  if (prefix_tokens > INT_MAX || nh > INT_MAX) return PA_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prefix_tokens == 0)   // nothing shared: plain varlen attention
    return from_cuda(pa::launch_varlen_tc(
        varlen_launch(q, kv_cache, block_table, query_start_loc, seq_lens, max_query_len, shape,
                      scale, causal ? 1 : 0, 0, out, lse),
        st));
  const int slots = num_prefix_splits + num_suffix_splits;
  {
    // Pass 1: every query row of the batch against the shared prefix (read
    // through row 0 of the table), no mask, cut into num_prefix_splits
    // pieces: slots [0, num_prefix_splits).
    pa::VarlenLaunch L = varlen_launch(q, kv_cache, block_table, query_start_loc, seq_lens,
                                       max_query_len, shape, scale, 0, 0, out, lse);
    L.virt_total_q = total_q;
    L.virt_seq = static_cast<int>(prefix_tokens);
    L.ws = workspace;
    L.ws_slots = slots;
    L.ws_slot0 = 0;
    L.kv_splits = num_prefix_splits;
    const long long per = (prefix_tokens + num_prefix_splits - 1) / num_prefix_splits;
    L.kv_chunk = static_cast<int>((per + 127) / 128 * 128);
    if (pa::launch_varlen_tc(L, st) != cudaSuccess) return PA_ERR_CUDA;
  }
  // Pass 2: each request against its own blocks after the prefix (positions
  // shift alike for keys and queries, so the call's mask is kept), cut into
  // num_suffix_splits pieces: slots [num_prefix_splits, slots).  A batch of
  // one query per request takes the split-KV decode kernel.
  const int suffix_max = static_cast<int>(std::max(0LL, max_seq_len - prefix_tokens));
  if (max_query_len == 1 && total_q == shape->num_seqs) {
    const pa::DecodeExt ext{num_common_prefix_blocks, static_cast<int>(prefix_tokens), slots,
                            num_prefix_splits};
    if (pa::launch_decode_splitkv(
            q, kv_cache, block_table, seq_lens, shape->num_seqs, shape->num_q_heads,
            shape->num_kv_heads, shape->head_size, shape->block_size, shape->num_blocks,
            shape->max_blocks_per_seq, scale, num_suffix_splits,
            static_cast<int>(pa::split_chunk(suffix_max, num_suffix_splits, shape->block_size)),
            workspace, device_error_ptr(), st, &ext) != cudaSuccess)
      return PA_ERR_CUDA;
  } else {
    pa::VarlenLaunch L2 = varlen_launch(q, kv_cache, block_table, query_start_loc, seq_lens,
                                        max_query_len, shape, scale, causal ? 1 : 0, 0, out, lse);
    L2.table_col0 = num_common_prefix_blocks;
    L2.seq_off = static_cast<int>(prefix_tokens);
    L2.ws = workspace;
    L2.ws_slots = slots;
    L2.ws_slot0 = num_prefix_splits;
    L2.kv_splits = num_suffix_splits;
    const long long per = (static_cast<long long>(suffix_max) + num_suffix_splits - 1) /
                          num_suffix_splits;
    L2.kv_chunk = static_cast<int>(std::max(128LL, (per + 127) / 128 * 128));
    if (pa::launch_varlen_tc(L2, st) != cudaSuccess) return PA_ERR_CUDA;
  }
  // Merge the partials by their LSE (the split-KV stage 2).
  return from_cuda(pa::launch_lse_merge(workspace, static_cast<int>(nh), slots,
                                        shape->head_size, out, lse, st));
}

int pa_device_sm_count(void) {
  static std::mutex mu;
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev < 64) cached[dev] = sms;
  return sms;
}

int pa_num_kv_splits(int max_seq_len, int sm_count) {
  if (sm_count <= 0) sm_count = pa_device_sm_count();
  if (sm_count <= 0) sm_count = 1;
  const long long by_len = (static_cast<long long>(max_seq_len > 0 ? max_seq_len : 0) + 511) / 512;
  long long s = by_len < 2LL * sm_count ? by_len : 2LL * sm_count;
  if (s < 1) s = 1;
  if (s > kMaxSplits) s = kMaxSplits;
  return static_cast<int>(s);
}

int pa_decode_num_kv_splits(int num_seqs, int num_kv_heads, int max_seq_len, int sm_count) {
  if (num_seqs <= 0 || num_kv_heads <= 0) return 1;
  if (sm_count <= 0) sm_count = pa_device_sm_count();
  if (sm_count <= 0) sm_count = 1;
  const long long units = static_cast<long long>(num_seqs) * num_kv_heads;
  long long s = (12LL * sm_count + units - 1) / units;
  const int page = pa_num_kv_splits(max_seq_len, sm_count);
  if (s > page) s = page;
  if (s < 1) s = 1;
  return static_cast<int>(s);
}

int pa_mla_num_kv_splits(int batch, int num_heads, int max_seq_len, int sm_count) {
  if (batch <= 0 || num_heads <= 0) return 1;
  if (sm_count <= 0) sm_count = pa_device_sm_count();
  if (sm_count <= 0) sm_count = 1;
  const long long units = static_cast<long long>(batch) * ((num_heads + 127) / 128);
  const long long pairs = sm_count / 2 > 0 ? sm_count / 2 : 1;
  long long s = (pairs + units - 1) / units;
  const long long by_len = (static_cast<long long>(max_seq_len > 0 ? max_seq_len : 0) + 511) / 512;
  if (s > by_len) s = by_len;
  if (s < 1) s = 1;
  if (s > kMaxSplits) s = kMaxSplits;
  return static_cast<int>(s);
}

size_t pa_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_splits, int dv) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_splits <= 0 || dv <= 0) return 0;
  return static_cast<size_t>(num_seqs) * num_q_heads * num_splits * (static_cast<size_t>(dv) + 1) *
         sizeof(float);
}

pa_status pa_decode_splitkv(const void* q, const void* kv_cache, const int32_t* block_table,
                            const int32_t* seq_lens, const pa_shape* shape, float scale,
                            int num_splits, int max_seq_len, float* workspace, void* stream) {
  if (!shape_ok(shape) || num_splits < 1 || num_splits > kMaxSplits || max_seq_len < 0)
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 16) return PA_ERR_UNSUPPORTED;
  if (shape->num_seqs == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr ||
      workspace == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 4) || !aligned(kv_cache, 16) || !aligned(workspace, 4)) return PA_ERR_INVALID;
  return from_cuda(pa::launch_decode_splitkv(
      q, kv_cache, block_table, seq_lens, shape->num_seqs, shape->num_q_heads,
      shape->num_kv_heads, shape->head_size, shape->block_size, shape->num_blocks,
      shape->max_blocks_per_seq, scale, num_splits,
      static_cast<int>(pa::split_chunk(max_seq_len, num_splits, shape->block_size)), workspace,
      device_error_ptr(),
      static_cast<cudaStream_t>(stream)));
}

pa_status pa_reshape_and_cache_fp8(const void* key, const void* value, void* kv_cache,
                                   const int64_t* slot_mapping, int num_tokens,
                                   const pa_shape* shape, float k_scale, float v_scale,
                                   void* stream) {
  if (shape == nullptr || num_tokens < 0) return PA_ERR_INVALID;
  if (shape->num_kv_heads <= 0 || shape->head_size <= 0 || shape->block_size <= 0 ||
      shape->block_size % 16 != 0 || shape->num_blocks <= 0)
    return PA_ERR_INVALID;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID;
  if (shape->head_size % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (key == nullptr || value == nullptr || kv_cache == nullptr || slot_mapping == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_reshape_and_cache_fp8(
      key, value, kv_cache, slot_mapping, num_tokens, shape->num_kv_heads, shape->head_size,
      shape->block_size, shape->num_blocks, k_scale, v_scale, device_error_ptr(),
      static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_splitkv_fp8(const void* q, const void* kv_cache, const int32_t* block_table,
                                const int32_t* seq_lens, const pa_shape* shape, float scale,
                                float k_scale, float v_scale, int num_splits, int max_seq_len,
                                float* workspace, void* stream) {
  if (!shape_ok(shape) || num_splits < 1 || num_splits > kMaxSplits || max_seq_len < 0)
    return PA_ERR_INVALID;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 16) return PA_ERR_UNSUPPORTED;
  if (shape->num_seqs == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr ||
      workspace == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 4) || !aligned(kv_cache, 16) || !aligned(workspace, 4)) return PA_ERR_INVALID;
  return from_cuda(pa::launch_decode_splitkv_fp8(
      q, kv_cache, block_table, seq_lens, shape->num_seqs, shape->num_q_heads,
      shape->num_kv_heads, shape->head_size, shape->block_size, shape->num_blocks,
      shape->max_blocks_per_seq, scale, k_scale, v_scale, num_splits,
      static_cast<int>(pa::split_chunk(max_seq_len, num_splits, shape->block_size)), workspace,
      device_error_ptr(), static_cast<cudaStream_t>(stream)));
}

static pa_status decode_window(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* seq_lens, const pa_shape* shape, float scale,
                               bool fp8, float k_scale, float v_scale, int sliding_window,
                               int num_sinks, void* out, float* lse, void* stream) {
  if (!shape_ok(shape) || sliding_window < 1 || num_sinks < 0 ||
      !logit_scale_ok(scale, k_scale) || !scale_ok(v_scale))
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 16) return PA_ERR_UNSUPPORTED;
  if (shape->num_seqs == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr ||
      out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 4) || !aligned(kv_cache, 16) || !aligned(out, 2) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return PA_ERR_INVALID;
  pa::DecodeWindowLaunch n{};
  n.q = q;
  n.cache = kv_cache;
  n.block_table = block_table;
  n.seq_lens = seq_lens;
  n.N = shape->num_seqs;
  n.Hq = shape->num_q_heads;
  n.Hkv = shape->num_kv_heads;
  n.d = shape->head_size;
  n.bs = shape->block_size;
  n.num_blocks = shape->num_blocks;
  n.max_blocks = shape->max_blocks_per_seq;
  n.window = sliding_window;
  n.sinks = num_sinks;
  n.scale = scale;
  n.k_scale = k_scale;
  n.v_scale = v_scale;
  n.fp8 = fp8;
  n.out = out;
  n.lse = lse;
  n.err = device_error_ptr();
  n.sm_count = pa_device_sm_count();
  if (n.sm_count <= 0) return PA_ERR_CUDA;
  return from_cuda(pa::launch_decode_window(n, static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_window(const void* q, const void* kv_cache, const int32_t* block_table,
                           const int32_t* seq_lens, const pa_shape* shape, float scale,
                           int sliding_window, int num_sinks, void* out, float* lse,
                           void* stream) {
  return decode_window(q, kv_cache, block_table, seq_lens, shape, scale, false, 1.f, 1.f,
                       sliding_window, num_sinks, out, lse, stream);
}

pa_status pa_decode_window_fp8(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* seq_lens, const pa_shape* shape, float scale,
                               float k_scale, float v_scale, int sliding_window, int num_sinks,
                               void* out, float* lse, void* stream) {
  return decode_window(q, kv_cache, block_table, seq_lens, shape, scale, true, k_scale, v_scale,
                       sliding_window, num_sinks, out, lse, stream);
}

pa_status pa_reshape_and_cache_fp4(const void* key, const void* value, int64_t key_stride,
                                   int64_t value_stride, void* kv_cache,
                                   const int64_t* slot_mapping, int num_tokens,
                                   const pa_shape* shape, float k_scale, float v_scale,
                                   void* stream) {
  if (shape == nullptr || num_tokens < 0 || shape->num_kv_heads <= 0 ||
      shape->num_kv_heads > kMaxGridYZ || shape->head_size <= 0 || shape->block_size <= 0 ||
      shape->block_size % 16 != 0 || shape->num_blocks <= 0)
    return PA_ERR_INVALID;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(shape->num_kv_heads) * shape->head_size;
  if (key_stride < width || value_stride < width || key_stride % 8 != 0 || value_stride % 8 != 0)
    return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (key == nullptr || value == nullptr || kv_cache == nullptr || slot_mapping == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_cache_write_fp4(
      key, value, key_stride, value_stride, kv_cache, slot_mapping, num_tokens,
      shape->num_kv_heads, shape->head_size, shape->block_size, shape->num_blocks, k_scale, v_scale,
      device_error_ptr(), static_cast<cudaStream_t>(stream)));
}

// Workspace of a decode call: the splits' partials, then (with sums) the logits.
static size_t partial_bytes(int num_seqs, int num_q_heads, int splits, int d) {
  const size_t n = static_cast<size_t>(num_seqs) * num_q_heads * splits * (d + 1) * 4;
  return (n + 15) / 16 * 16;
}
static bool workspace_args_ok(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                              int max_seq_len) {
  return num_seqs >= 0 && num_q_heads > 0 && num_kv_heads > 0 && head_size > 0 && max_seq_len >= 0;
}
// (152 where there is no device to ask, as when a size is planned beforehand.)
static int sm_count_or_default() {
  const int n = pa_device_sm_count();
  return n > 0 ? n : 152;
}

size_t pa_decode_fp4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_size, int max_seq_len, int with_scores) {
  if (!workspace_args_ok(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len)) return 0;
  return pa::decode_fp4_workspace(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len,
                                  with_scores != 0, sm_count_or_default())
      .bytes;
}

size_t pa_decode_scores_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                        int head_size, int max_seq_len) {
  if (!workspace_args_ok(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len)) return 0;
  const int S = pa_decode_num_kv_splits(num_seqs, num_kv_heads, max_seq_len, sm_count_or_default());
  return partial_bytes(num_seqs, num_q_heads, S, head_size) +
         static_cast<size_t>(num_seqs) * num_q_heads * max_seq_len * 4;
}

// Checks that the decode calls below share; PA_OK with *done where there is nothing to do.
static pa_status decode_args(const void* q, const void* kv_cache, const int32_t* block_table,
                             const int32_t* seq_lens, const pa_shape* shape, float scale,
                             float k_scale, float v_scale, int max_seq_len, const void* out,
                             const float* lse, bool* done) {
  *done = false;
  if (!shape_ok(shape) || max_seq_len < 0 || !logit_scale_ok(scale, k_scale) || !scale_ok(v_scale))
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_q_heads / shape->num_kv_heads > 16) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(shape->num_seqs) * shape->num_q_heads > INT_MAX) return PA_ERR_INVALID;
  if (shape->num_seqs == 0) {
    *done = true;
    return PA_OK;
  }
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr ||
      out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 4) || !aligned(kv_cache, 16) || !aligned(out, 2) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return PA_ERR_INVALID;
  return PA_OK;
}

static pa_status decode_fp4(const void* q, const void* kv_cache, const int32_t* block_table,
                            const int32_t* seq_lens, const pa_shape* shape, float scale,
                            float k_scale, float v_scale, int max_seq_len, void* workspace,
                            size_t workspace_bytes, bool with_scores, float* scores,
                            int score_tokens, void* out, float* lse, void* stream) {
  bool done;
  const pa_status s = decode_args(q, kv_cache, block_table, seq_lens, shape, scale, k_scale,
                                  v_scale, max_seq_len, out, lse, &done);
  if (s != PA_OK || done) return s;
  if (with_scores && (scores == nullptr || !aligned(scores, 4) || score_tokens < max_seq_len))
    return PA_ERR_INVALID;
  const size_t need =
      pa_decode_fp4_workspace_bytes(shape->num_seqs, shape->num_q_heads, shape->num_kv_heads,
                                    shape->head_size, max_seq_len, with_scores);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return PA_ERR_INVALID;
  pa::DecodeFp4Launch n{};
  n.q = q;
  n.cache = kv_cache;
  n.block_table = block_table;
  n.seq_lens = seq_lens;
  n.N = shape->num_seqs;
  n.Hq = shape->num_q_heads;
  n.Hkv = shape->num_kv_heads;
  n.d = shape->head_size;
  n.bs = shape->block_size;
  n.num_blocks = shape->num_blocks;
  n.max_blocks = shape->max_blocks_per_seq;
  n.scale = scale;
  n.k_scale = k_scale;
  n.v_scale = v_scale;
  n.max_seq_len = max_seq_len;
  n.workspace = workspace;
  n.scores = scores;
  n.score_tokens = score_tokens;
  n.out = out;
  n.lse = lse;
  n.err = device_error_ptr();
  n.sm_count = sm_count_or_default();
  return from_cuda(pa::launch_decode_fp4(n, static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_fp4(const void* q, const void* kv_cache, const int32_t* block_table,
                        const int32_t* seq_lens, const pa_shape* shape, float scale, float k_scale,
                        float v_scale, int max_seq_len, void* workspace, size_t workspace_bytes,
                        void* out, float* lse, void* stream) {
  return decode_fp4(q, kv_cache, block_table, seq_lens, shape, scale, k_scale, v_scale, max_seq_len,
                    workspace, workspace_bytes, false, nullptr, 0, out, lse, stream);
}

pa_status pa_decode_scores_fp4(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* seq_lens, const pa_shape* shape, float scale,
                               float k_scale, float v_scale, int max_seq_len, void* workspace,
                               size_t workspace_bytes, float* scores, int score_tokens, void* out,
                               float* lse, void* stream) {
  return decode_fp4(q, kv_cache, block_table, seq_lens, shape, scale, k_scale, v_scale, max_seq_len,
                    workspace, workspace_bytes, true, scores, score_tokens, out, lse, stream);
}

pa_status pa_decode_scores(const void* q, const void* kv_cache, const int32_t* block_table,
                           const int32_t* seq_lens, const pa_shape* shape, float scale,
                           int max_seq_len, void* workspace, size_t workspace_bytes, float* scores,
                           int score_tokens, void* out, float* lse, void* stream) {
  bool done;
  const pa_status s = decode_args(q, kv_cache, block_table, seq_lens, shape, scale, 1.f, 1.f,
                                  max_seq_len, out, lse, &done);
  if (s != PA_OK || done) return s;
  if (scores == nullptr || !aligned(scores, 4) || score_tokens < max_seq_len) return PA_ERR_INVALID;
  const size_t need =
      pa_decode_scores_workspace_bytes(shape->num_seqs, shape->num_q_heads, shape->num_kv_heads,
                                       shape->head_size, max_seq_len);
  if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
    return PA_ERR_INVALID;
  const int S = pa_decode_num_kv_splits(shape->num_seqs, shape->num_kv_heads, max_seq_len,
                                        sm_count_or_default());
  float* ws = static_cast<float*>(workspace);
  pa::DecodeExt x{0, 0, S, 0};
  x.logits = reinterpret_cast<float*>(
      static_cast<char*>(workspace) +
      partial_bytes(shape->num_seqs, shape->num_q_heads, S, shape->head_size));
  x.logit_tokens = max_seq_len;
  const cudaError_t e = pa::launch_decode_splitkv(
      q, kv_cache, block_table, seq_lens, shape->num_seqs, shape->num_q_heads,
      shape->num_kv_heads, shape->head_size, shape->block_size, shape->num_blocks,
      shape->max_blocks_per_seq, scale, S,
      static_cast<int>(pa::split_chunk(max_seq_len, S, shape->block_size)), ws, device_error_ptr(),
      static_cast<cudaStream_t>(stream), &x);
  if (e != cudaSuccess) return from_cuda(e);
  pa::ScoresLaunch m{};
  m.ws = ws;
  m.S = S;
  m.out_scale = 1.f;
  m.logits = x.logits;
  m.logit_tokens = max_seq_len;
  m.seq_lens = seq_lens;
  m.N = shape->num_seqs;
  m.Hq = shape->num_q_heads;
  m.Hkv = shape->num_kv_heads;
  m.d = shape->head_size;
  m.max_seq_len = max_seq_len;
  m.scores = scores;
  m.score_tokens = score_tokens;
  m.out = out;
  m.lse = lse;
  m.err = device_error_ptr();
  return from_cuda(pa::launch_decode_scores(m, static_cast<cudaStream_t>(stream)));
}

static pa_status evict(void* kv_cache, const pa_shape* shape, bool four, int element_bytes,
                       const int32_t* block_table, const int32_t* seq_lens, const float* scores,
                       int score_tokens, int budget, int num_recent, int num_first,
                       int32_t* new_lens, float* new_scores, int32_t* kept, int32_t* free_blocks,
                       int num_free, const int32_t* free_start, int32_t* new_free_start,
                       void* stream) {
  if (!shape_ok(shape) || score_tokens <= 0 || budget < 1 || budget > (1 << 30) ||
      num_recent < 0 || num_first < 0 || num_recent > budget || num_first > budget - num_recent ||
      num_free < 0 || (!four && element_bytes != 1 && element_bytes != 2))
    return PA_ERR_INVALID;
  if (shape->head_size != 64 && shape->head_size != 128) return PA_ERR_UNSUPPORTED;
  if (shape->num_seqs == 0) return PA_OK;
  if (kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr || scores == nullptr ||
      new_lens == nullptr || new_scores == nullptr || kept == nullptr)
    return PA_ERR_INVALID;
  // A free list comes with its two ends, or not at all.
  if ((free_blocks == nullptr) != (free_start == nullptr) ||
      (free_blocks == nullptr) != (new_free_start == nullptr))
    return PA_ERR_INVALID;
  if (!aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(scores, 4) || !aligned(new_lens, 4) || !aligned(new_scores, 4) ||
      !aligned(kept, 4) || !aligned(free_blocks, 4) || !aligned(free_start, 4) ||
      !aligned(new_free_start, 4))
    return PA_ERR_INVALID;
  // Inputs, then outputs.  Lengths, sums and the list's start may be updated in place.
  const size_t n4 = static_cast<size_t>(shape->num_seqs) * 4;
  const size_t units4 = n4 * shape->num_kv_heads, one = free_start != nullptr ? 4u : 0u;
  const Range ranges[] = {{block_table, n4 * shape->max_blocks_per_seq},
                          {seq_lens, n4},
                          {scores, units4 * score_tokens},
                          {free_start, one},
                          {new_lens, n4},
                          {new_scores, units4 * score_tokens},
                          {kept, units4 * budget},
                          {free_blocks, static_cast<size_t>(num_free) * 4},
                          {new_free_start, one}};
  const size_t row = four ? shape->head_size / 16 * 9 : shape->head_size * element_bytes;
  const Range pool{kv_cache, static_cast<size_t>(shape->num_blocks) * shape->num_kv_heads *
                                 shape->block_size * 2 * row};
  for (const Range& r : ranges)
    if (overlap(pool, r)) return PA_ERR_INVALID;
  for (int out = 4; out < 9; ++out)
    for (int k = 0; k < out; ++k) {
      const bool same = (out == 4 && k == 1) || (out == 5 && k == 2) || (out == 8 && k == 3);
      if (same && ranges[out].p == ranges[k].p) continue;
      if (overlap(ranges[out], ranges[k])) return PA_ERR_INVALID;
    }
  pa::EvictLaunch n{};
  n.cache = kv_cache;
  n.block_table = block_table;
  n.seq_lens = seq_lens;
  n.scores = scores;
  n.new_scores = new_scores;
  n.new_lens = new_lens;
  n.kept = kept;
  n.free_blocks = free_blocks;
  n.free_start = free_start;
  n.new_free_start = new_free_start;
  n.num_free = num_free;
  n.N = shape->num_seqs;
  n.Hkv = shape->num_kv_heads;
  n.d = shape->head_size;
  n.bs = shape->block_size;
  n.num_blocks = shape->num_blocks;
  n.max_blocks = shape->max_blocks_per_seq;
  n.score_tokens = score_tokens;
  n.budget = budget;
  n.recent = num_recent;
  n.first = num_first;
  n.four = four;
  n.row_bytes = shape->head_size * element_bytes;
  n.err = device_error_ptr();
  return from_cuda(pa::launch_evict(n, static_cast<cudaStream_t>(stream)));
}

pa_status pa_evict(void* kv_cache, const pa_shape* shape, int element_bytes,
                   const int32_t* block_table, const int32_t* seq_lens, const float* scores,
                   int score_tokens, int budget, int num_recent, int num_first, int32_t* new_lens,
                   float* new_scores, int32_t* kept, int32_t* free_blocks, int num_free,
                   const int32_t* free_start, int32_t* new_free_start, void* stream) {
  return evict(kv_cache, shape, false, element_bytes, block_table, seq_lens, scores, score_tokens,
               budget, num_recent, num_first, new_lens, new_scores, kept, free_blocks, num_free,
               free_start, new_free_start, stream);
}

pa_status pa_evict_fp4(void* kv_cache, const pa_shape* shape, const int32_t* block_table,
                       const int32_t* seq_lens, const float* scores, int score_tokens, int budget,
                       int num_recent, int num_first, int32_t* new_lens, float* new_scores,
                       int32_t* kept, int32_t* free_blocks, int num_free,
                       const int32_t* free_start, int32_t* new_free_start, void* stream) {
  return evict(kv_cache, shape, true, 0, block_table, seq_lens, scores, score_tokens, budget,
               num_recent, num_first, new_lens, new_scores, kept, free_blocks, num_free, free_start,
               new_free_start, stream);
}

pa_status pa_plan_step(const int32_t* context_lens, const int32_t* query_lens,
                       const int32_t* free_blocks, const int32_t* free_start, int num_free,
                       int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks,
                       int max_tokens, int32_t* block_table, int32_t* query_start_loc,
                       int32_t* seq_lens, int32_t* positions, int64_t* slot_mapping,
                       int32_t* totals, void* stream) {
  if (num_free < 0 || num_seqs < 0 || num_seqs > kMaxGridYZ || max_blocks_per_seq <= 0 ||
      block_size <= 0 || block_size % 16 != 0 || num_blocks <= 0 || max_tokens < 0)
    return PA_ERR_INVALID;
  if (query_start_loc == nullptr || totals == nullptr ||
      (num_seqs > 0 && (context_lens == nullptr || query_lens == nullptr ||
                        block_table == nullptr || seq_lens == nullptr)) ||
      (num_free > 0 && free_blocks == nullptr) ||
      (max_tokens > 0 && (positions == nullptr || slot_mapping == nullptr)))
    return PA_ERR_INVALID;
  if (!aligned(context_lens, 4) || !aligned(query_lens, 4) || !aligned(free_blocks, 4) ||
      !aligned(free_start, 4) || !aligned(block_table, 4) || !aligned(query_start_loc, 4) ||
      !aligned(seq_lens, 4) || !aligned(positions, 4) || !aligned(slot_mapping, 8) ||
      !aligned(totals, 4))
    return PA_ERR_INVALID;
  // Inputs, then outputs: a CTA reads inputs while another writes its outputs.
  const size_t n4 = static_cast<size_t>(num_seqs) * 4, cap = static_cast<size_t>(max_tokens);
  const Range ranges[] = {
      {context_lens, n4}, {query_lens, n4}, {free_blocks, static_cast<size_t>(num_free) * 4},
      {free_start, free_start != nullptr ? 4u : 0u}, {block_table, n4 * max_blocks_per_seq},
      {query_start_loc, n4 + 4}, {seq_lens, n4}, {positions, cap * 4}, {slot_mapping, cap * 8},
      {totals, 8}};
  for (int out = 4; out < 10; ++out)
    for (int k = 0; k < out; ++k)
      if (overlap(ranges[out], ranges[k])) return PA_ERR_INVALID;
  return from_cuda(pa::launch_plan_step(
      context_lens, query_lens, free_blocks, free_start, num_free, num_seqs, max_blocks_per_seq,
      block_size, num_blocks, max_tokens, block_table, query_start_loc, seq_lens, positions,
      slot_mapping, totals, device_error_ptr(), static_cast<cudaStream_t>(stream)));
}

static pa_status norm_rope(const void* q, const void* key, const void* value, int64_t q_stride,
                           int64_t key_stride, int64_t value_stride, const void* q_weight,
                           const void* k_weight, float eps, const float* cos_sin,
                           int max_position, int rotary_dim, int interleaved,
                           const int32_t* positions, void* kv_cache, const int64_t* slot_mapping,
                           int num_tokens, const pa_shape* shape, bool fp8, float k_scale,
                           float v_scale, void* q_out, void* stream) {
  if (shape == nullptr || num_tokens < 0 || shape->num_q_heads <= 0 || shape->num_kv_heads <= 0 ||
      shape->num_q_heads > kMaxGridYZ || shape->num_kv_heads > kMaxGridYZ ||
      shape->head_size <= 0 || shape->block_size <= 0 || shape->block_size % 16 != 0 ||
      shape->num_blocks <= 0 || rotary_dim < 0 || rotary_dim > shape->head_size ||
      !(eps >= 0.f && eps <= 3.4028234663852886e38f))
    return PA_ERR_INVALID;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID;
  if ((shape->head_size != 64 && shape->head_size != 128) || rotary_dim % 16 != 0)
    return PA_ERR_UNSUPPORTED;
  const int64_t qw = static_cast<int64_t>(shape->num_q_heads) * shape->head_size;
  const int64_t kw = static_cast<int64_t>(shape->num_kv_heads) * shape->head_size;
  if (q_stride < qw || key_stride < kw || value_stride < kw || q_stride % 8 != 0 ||
      key_stride % 8 != 0 || value_stride % 8 != 0)
    return PA_ERR_INVALID;
  if (rotary_dim > 0 && max_position <= 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (q == nullptr || key == nullptr || value == nullptr || kv_cache == nullptr ||
      slot_mapping == nullptr || q_out == nullptr || (q_weight == nullptr) != (k_weight == nullptr) ||
      (rotary_dim > 0 && (cos_sin == nullptr || positions == nullptr)))
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(cos_sin, 16) || !aligned(kv_cache, 16) ||
      !aligned(q_out, 16) || !aligned(positions, 4) || !aligned(slot_mapping, 8))
    return PA_ERR_INVALID;
  // q_out is q (dense) or lies apart from all three inputs.
  auto rows = [&](const void* p, int64_t stride, int64_t width) {
    return Range{p, static_cast<size_t>((num_tokens - 1) * stride + width) * 2};   // bf16
  };
  const Range out = rows(q_out, qw, qw);
  if ((q_out == q ? q_stride != qw && num_tokens > 1 : overlap(out, rows(q, q_stride, qw))) ||
      overlap(out, rows(key, key_stride, kw)) || overlap(out, rows(value, value_stride, kw)))
    return PA_ERR_INVALID;
  pa::NormRopeLaunch n{};
  n.q = q;
  n.key = key;
  n.value = value;
  n.q_stride = q_stride;
  n.key_stride = key_stride;
  n.value_stride = value_stride;
  n.q_weight = q_weight;
  n.k_weight = k_weight;
  n.eps = eps;
  n.cos_sin = cos_sin;
  n.max_position = max_position;
  n.rotary_dim = rotary_dim;
  n.interleaved = interleaved ? 1 : 0;
  n.positions = positions;
  n.cache = kv_cache;
  n.slot_mapping = slot_mapping;
  n.num_tokens = num_tokens;
  n.Hq = shape->num_q_heads;
  n.Hkv = shape->num_kv_heads;
  n.d = shape->head_size;
  n.bs = shape->block_size;
  n.num_blocks = shape->num_blocks;
  n.fp8 = fp8;
  n.k_scale = k_scale;
  n.v_scale = v_scale;
  n.q_out = q_out;
  n.err = device_error_ptr();
  n.sm_count = pa_device_sm_count();
  if (n.sm_count <= 0) return PA_ERR_CUDA;
  return from_cuda(pa::launch_norm_rope(n, static_cast<cudaStream_t>(stream)));
}

pa_status pa_qk_norm_rope_cache(const void* q, const void* key, const void* value,
                                int64_t q_stride, int64_t key_stride, int64_t value_stride,
                                const void* q_weight, const void* k_weight, float eps,
                                const float* cos_sin, int max_position, int rotary_dim,
                                int interleaved, const int32_t* positions, void* kv_cache,
                                const int64_t* slot_mapping, int num_tokens,
                                const pa_shape* shape, void* q_out, void* stream) {
  return norm_rope(q, key, value, q_stride, key_stride, value_stride, q_weight, k_weight, eps,
                   cos_sin, max_position, rotary_dim, interleaved, positions, kv_cache,
                   slot_mapping, num_tokens, shape, false, 1.f, 1.f, q_out, stream);
}

pa_status pa_qk_norm_rope_cache_fp8(const void* q, const void* key, const void* value,
                                    int64_t q_stride, int64_t key_stride, int64_t value_stride,
                                    const void* q_weight, const void* k_weight, float eps,
                                    const float* cos_sin, int max_position, int rotary_dim,
                                    int interleaved, const int32_t* positions, void* kv_cache,
                                    const int64_t* slot_mapping, int num_tokens,
                                    const pa_shape* shape, float k_scale, float v_scale,
                                    void* q_out, void* stream) {
  return norm_rope(q, key, value, q_stride, key_stride, value_stride, q_weight, k_weight, eps,
                   cos_sin, max_position, rotary_dim, interleaved, positions, kv_cache,
                   slot_mapping, num_tokens, shape, true, k_scale, v_scale, q_out, stream);
}

pa_status pa_lse_merge(const float* workspace, int num_seqs, int num_q_heads, int num_splits,
                       int dv, void* out, float* lse, void* stream) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_splits < 1 || num_splits > kMaxSplits || dv <= 0)
    return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (workspace == nullptr || out == nullptr) return PA_ERR_INVALID;
  if (!aligned(workspace, 4) || !aligned(out, 2) || !aligned(lse, 4)) return PA_ERR_INVALID;
  const long long nh = static_cast<long long>(num_seqs) * num_q_heads;
  if (nh > INT_MAX) return PA_ERR_INVALID;
  return from_cuda(pa::launch_lse_merge(workspace, static_cast<int>(nh), num_splits, dv, out, lse,
                                        static_cast<cudaStream_t>(stream)));
}

pa_status pa_mla_decode(const void* q, const void* kv_cache, const int32_t* block_table,
                        const int32_t* seq_lens, int batch, int num_heads, int kv_lora_rank,
                        int rope_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                        int max_seq_len, float scale, int num_splits, float* workspace, void* out,
                        float* lse,
                        void* stream) {
  if (batch < 0 || num_heads <= 0 || kv_lora_rank <= 0 || rope_dim < 0 || block_size <= 0 ||
      block_size % 16 != 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || num_splits < 1 ||
      num_splits > kMaxSplits || batch > kMaxGridYZ || num_splits > kMaxGridYZ || max_seq_len < 0)
    return PA_ERR_INVALID;
  if (kv_lora_rank != 512 || rope_dim != 64 || num_heads % 64 != 0 || block_size % 32 != 0)
    return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (q == nullptr || kv_cache == nullptr || block_table == nullptr || seq_lens == nullptr ||
      workspace == nullptr || out == nullptr)
    return PA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(workspace, 4) || !aligned(out, 2) ||
      !aligned(lse, 4))
    return PA_ERR_INVALID;
  return from_cuda(pa::launch_mla_tc(q, kv_cache, block_table, seq_lens, batch, num_heads,
                                         block_size, num_blocks, max_blocks_per_seq, scale,
                                         num_splits,
                                         static_cast<int>(pa::split_chunk(max_seq_len, num_splits,
                                                                          block_size)),
                                         workspace, out, lse, device_error_ptr(),
                                         static_cast<cudaStream_t>(stream)));
}

const char* pa_status_string(pa_status status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID: return "PA_ERR_INVALID: invalid argument";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: configuration not built";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: CUDA launch or query failed";
  }
  return "unknown pa_status";
}

pa_status pa_get_device_error(int* code, void* stream) {
  if (code == nullptr) return PA_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return PA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, pa::g_device_error, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(pa::g_device_error, &zero, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
  *code = v;
  return PA_OK;
}

}  // extern "C"
