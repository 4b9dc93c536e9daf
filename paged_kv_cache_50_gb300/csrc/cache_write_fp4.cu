// The quantising cache write into a 4-bit pool (layout: fp4.cuh).
//
// For each 16 elements x of a token's head row, with the layer's scale k:
//   s = e4m3(min(448, max|x| / k / 6)),  t = fl32(s k),  code = e2m1(x / t)
// (quotients in fp32 with IEEE rounding, conversions to nearest even, codes
// saturating at +-6; t == 0: codes 0).  A NaN makes the block's scale NaN.  6 is the
// largest code, so that a block's largest element keeps the most digits.
//
// One thread turns 16 elements of a key, and the value's, into 8 bytes of codes and one
// scale each.  A batch of 18432 tokens of 8 heads of 128 (97 MB) takes 18 us (with one
// block of 16 for each thread: 29); a decode step's is bound by its launch.
#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

// (x, y) = -(x, y) / t, correctly rounded: one step of Markstein's correction
// ("Computation of elementary functions on the IBM RISC System/6000 processor", 1990)
// from r = -fl(1 / t), while t, r and the quotient stay away from the range's ends (a
// quotient that is too small rounds to the same code all the same).  The remainder of an
// exact quotient is +0, and +0 r = -0 leaves the sign of a zero as it is.
__device__ __forceinline__ void negative_quotients(float& x, float& y, float t, float r) {
  asm("{\n.reg .b64 x, t, r, q, e;\n"
      "mov.b64 x, {%0, %1};\nmov.b64 t, {%2, %2};\nmov.b64 r, {%3, %3};\n"
      "mul.rn.f32x2 q, x, r;\nfma.rn.f32x2 e, q, t, x;\nfma.rn.f32x2 q, e, r, q;\n"
      "mov.b64 {%0, %1}, q;\n}"
      : "+f"(x), "+f"(y)
      : "f"(t), "f"(r));
}

// n / by for n >= 0, without a division of 64 bits where 32 do.
__device__ __forceinline__ int64_t quotient(int64_t n, int by) {
  return n <= 0xffffffffLL ? static_cast<int64_t>(static_cast<uint32_t>(n) / static_cast<uint32_t>(by))
                           : n / by;
}

// Codes of -v.
__device__ __forceinline__ uint32_t pack8(const float* v) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w ^ 0x88888888u;
}

// Beyond this a scale and its reciprocal may leave the range of the steps below.
__device__ __forceinline__ bool ordinary(float t) { return t > 0x1p-80f && t < 0x1p80f; }

// 16 elements (w), the layer's scale and fl(1 / scale) -> their codes and their scale.
__device__ __forceinline__ uint2 quantised(const uint32_t (&w)[8], float step, float r_step,
                                           uint32_t& s8) {
  __nv_bfloat162 most = __habs2(reinterpret_cast<const __nv_bfloat162&>(w[0]));
#pragma unroll
  for (int k = 1; k < 8; ++k)
    most = __hmax2_nan(most, __habs2(reinterpret_cast<const __nv_bfloat162&>(w[k])));
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  const float top = __bfloat162float(__hmax_nan(most.x, most.y));
  // top / step / 6, both quotients by Markstein's step as above.  (What is cut off at
  // 2^20 saturates the scale all the same, what is too small for a step rounds to 0.)
  float a;
  if (ordinary(step)) {
    const float cut = fminf(top, 0x1p20f * step);
    a = cut * r_step;
    a = fmaf(fmaf(-a, step, cut), r_step, a);
  } else {
    a = fminf(__fdiv_rn(top, step), 0x1p20f);
  }
  const float sixth = 1.f / 6.f;
  float b = a * sixth;
  b = fmaf(fmaf(-b, 6.f, a), sixth, b);
  if (top != top) b = top;
  asm("{\n.reg .b16 s;\ncvt.rn.satfinite.e4m3x2.f32 s, %1, %2;\ncvt.u32.u16 %0, s;\n}"
      : "=r"(s8)
      : "f"(0.f), "f"(b));
  const float t = __low2float(__half2_raw{static_cast<unsigned short>(fp4::widen_scales(s8)), 0}) * step;
  if (!(t > 0.f)) return make_uint2(0u, 0u);   // (or NaN)
  if (ordinary(t) && top < 0x1p20f * t) {
    const float r = -__frcp_rn(t);
#pragma unroll
    for (int k = 0; k < 16; k += 2) negative_quotients(x[k], x[k + 1], t, r);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __fdiv_rn(x[k], -t);
  }
  return make_uint2(pack8(x), pack8(x + 8));
}

struct WriteArgs {
  const __nv_bfloat16* key;
  const __nv_bfloat16* value;
  uint8_t* cache;
  const int64_t* slot_mapping;
  int* err;
  int64_t key_stride, value_stride, blocks, num_slots, block_bytes;
  int row_blocks, row_log2, head_log2, bs, bs_log2;
  float k_scale, v_scale, k_inverse, v_inverse;
};

__global__ void __launch_bounds__(256) cache_write_fp4_kernel(const __grid_constant__ WriteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= a.blocks) return;
  // Block n: token, and which 16 elements of its row, of the key and of the value.
  const int64_t t = a.row_log2 >= 0 ? n >> a.row_log2 : quotient(n, a.row_blocks);
  const int b = static_cast<int>(n - t * a.row_blocks);
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (b == 0) record_error(a.err, PA_DEVERR_SLOT);
    return;
  }
  const uint4* key = reinterpret_cast<const uint4*>(a.key + t * a.key_stride + b * 16);
  const uint4* value = reinterpret_cast<const uint4*>(a.value + t * a.value_stride + b * 16);
  uint32_t k[8], v[8];
  *reinterpret_cast<uint4*>(k) = __ldcs(key);
  *reinterpret_cast<uint4*>(k + 4) = __ldcs(key + 1);
  *reinterpret_cast<uint4*>(v) = __ldcs(value);
  *reinterpret_cast<uint4*>(v + 4) = __ldcs(value + 1);
  const int64_t blk = a.bs_log2 >= 0 ? slot >> a.bs_log2 : quotient(slot, a.bs);
  const int off = static_cast<int>(slot - blk * a.bs);
  const int per_head = 1 << a.head_log2;   // blocks of 16 in a head row
  const int d = 16 * per_head, head = b >> a.head_log2, e = b & (per_head - 1), row = off & 15;
  uint8_t* tile = a.cache + blk * a.block_bytes +
                  static_cast<int64_t>(head * (a.bs >> 4) + (off >> 4)) * (2 * fp4::tile_bytes(d));
  uint8_t* codes = tile + row * (d / 2) + e * 8;
  uint8_t* scales = tile + 8 * d + row * per_head + e;
  uint32_t s8;
  *reinterpret_cast<uint2*>(codes) = quantised(k, a.k_scale, a.k_inverse, s8);
  *scales = static_cast<uint8_t>(s8);
  *reinterpret_cast<uint2*>(codes + fp4::tile_bytes(d)) = quantised(v, a.v_scale, a.v_inverse, s8);
  scales[fp4::tile_bytes(d)] = static_cast<uint8_t>(s8);
}

}  // namespace

cudaError_t launch_cache_write_fp4(const void* key, const void* value, int64_t key_stride,
                                   int64_t value_stride, void* cache, const int64_t* slot_mapping,
                                   int num_tokens, int num_kv_heads, int head_size, int block_size,
                                   int num_blocks, float k_scale, float v_scale, int* err,
                                   cudaStream_t stream) {
  WriteArgs a{};
  a.key = static_cast<const __nv_bfloat16*>(key);
  a.value = static_cast<const __nv_bfloat16*>(value);
  a.cache = static_cast<uint8_t*>(cache);
  a.slot_mapping = slot_mapping;
  a.err = err;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.row_blocks = num_kv_heads * head_size / 16;
  a.blocks = static_cast<int64_t>(num_tokens) * a.row_blocks;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.block_bytes = static_cast<int64_t>(num_kv_heads) * (block_size / 16) * 2 * fp4::tile_bytes(head_size);
  a.row_log2 = block_size_log2(a.row_blocks);
  a.head_log2 = block_size_log2(head_size / 16);
  a.bs = block_size;
  a.bs_log2 = block_size_log2(block_size);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_inverse = 1.f / k_scale;
  a.v_inverse = 1.f / v_scale;
  const int64_t ctas = (a.blocks + 255) / 256;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(cache_write_fp4_kernel, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream, a);
}

}  // namespace pa
