// The quantising cache write into a 4-bit pool (layout: fp4.cuh).
//
// For each 16 elements x of a token's head row, with the layer's scale k:
//   s = e4m3(min(448, max|x| / k / 6)),  t = fl32(s k),  code = e2m1(x / t)
// (quotients in fp32 with IEEE rounding, conversions to nearest even, codes
// saturating at +-6; t == 0: codes 0).  A NaN makes the block's scale NaN.  6 is the
// largest code, so that a block's largest element keeps the most digits.
//
// The code of x / t does not depend on the quotient's rounding: x has 8 significant
// bits, but the quotient is compared with the codes' midpoints m, so it matters
// only that fl32(x / t) equals m where x / t does, and lies on x / t's side of it
// where not.
//
// One thread turns 16 elements into 8 bytes of codes and one scale.  Bound by HBM
// for large batches, by the launch for small ones.
#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

// x / t, correctly rounded: one step of Markstein's correction ("Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990) from r = fl(1 /
// t), while t, r and the remainder stay in the normal range.  The sign is x's, also
// where x is a zero.
__device__ __forceinline__ float quotient(float x, float t, float r) {
  const float q = x * r;
  return copysignf(fmaf(fmaf(-q, t, x), r, q), x);
}

__device__ __forceinline__ uint32_t pack8(const float (&v)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(v[2 * k], v[2 * k + 1]),
                                                        __NV_E2M1, cudaRoundNearest))
         << (8 * k);
  return w;
}

__global__ void __launch_bounds__(256)
cache_write_fp4_kernel(const __nv_bfloat16* __restrict__ key, const __nv_bfloat16* __restrict__ value,
                       int64_t key_stride, int64_t value_stride, uint8_t* __restrict__ cache,
                       const int64_t* __restrict__ slot_mapping, int64_t blocks, int row_blocks,
                       int head_log2, int Hkv, int bs, int64_t num_slots, float k_scale,
                       float v_scale, int* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= blocks) return;
  // Block n: token, K or V, and which 16 elements of the token's row.
  const int64_t t = n / (2 * row_blocks);
  int b = static_cast<int>(n - t * (2 * row_blocks));
  const bool is_v = b >= row_blocks;
  if (is_v) b -= row_blocks;
  const int64_t slot = slot_mapping[t];
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (b == 0 && !is_v) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  const __nv_bfloat16* src =
      (is_v ? value + t * value_stride : key + t * key_stride) + static_cast<int64_t>(b) * 16;
  const uint4 lo = __ldcs(reinterpret_cast<const uint4*>(src));
  const uint4 hi = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float x[16];
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    top = fmaxf(top, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
    nan |= x[2 * k] != x[2 * k] || x[2 * k + 1] != x[2 * k + 1];
  }
  const float step = is_v ? v_scale : k_scale;
  const __nv_fp8_storage_t s8 =
      nan ? 0x7f
          : __nv_cvt_float_to_fp8(__fdiv_rn(__fdiv_rn(top, step), 6.f), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  const float tt = s * step;
  uint2 codes = make_uint2(0u, 0u);
  if (!nan && tt > 0.f) {
    float q[16];
    if (tt > 0x1p-80f && tt < 0x1p80f) {
      const float r = __frcp_rn(tt);
      const float lim = 8.f * tt;   // beyond it the code saturates all the same
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k] = quotient(fminf(fmaxf(x[k], -lim), lim), tt, r);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k] = __fdiv_rn(x[k], tt);
    }
    const float(&q0)[8] = reinterpret_cast<const float(&)[8]>(q[0]);
    const float(&q1)[8] = reinterpret_cast<const float(&)[8]>(q[8]);
    codes = make_uint2(pack8(q0), pack8(q1));
  }
  const int64_t blk = slot / bs;
  const int off = static_cast<int>(slot - blk * bs);
  const int per_head = 1 << head_log2;   // blocks of 16 in a head row
  const int d = 16 * per_head, head = b >> head_log2, e = b & (per_head - 1);
  uint8_t* tile = cache + fp4::pair_at(blk, head, off >> 4, Hkv, bs >> 4, d) +
                  (is_v ? fp4::tile_bytes(d) : 0);
  const int row = off & 15;
  *reinterpret_cast<uint2*>(tile + row * (d / 2) + e * 8) = codes;
  tile[8 * d + row * per_head + e] = s8;
}

}  // namespace

cudaError_t launch_cache_write_fp4(const void* key, const void* value, int64_t key_stride,
                                   int64_t value_stride, void* cache, const int64_t* slot_mapping,
                                   int num_tokens, int num_kv_heads, int head_size, int block_size,
                                   int num_blocks, float k_scale, float v_scale, int* err,
                                   cudaStream_t stream) {
  const int row_blocks = num_kv_heads * head_size / 16;
  const int64_t blocks = static_cast<int64_t>(num_tokens) * 2 * row_blocks;
  const int64_t ctas = (blocks + 255) / 256;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(cache_write_fp4_kernel, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream,
                    static_cast<const __nv_bfloat16*>(key),
                    static_cast<const __nv_bfloat16*>(value), key_stride, value_stride,
                    static_cast<uint8_t*>(cache), slot_mapping, blocks, row_blocks,
                    block_size_log2(head_size / 16), num_kv_heads, block_size,
                    static_cast<int64_t>(num_blocks) * block_size, k_scale, v_scale, err);
}

}  // namespace pa
