// What the tcgen05 attention kernels share: the swizzled tile layout, softmax
// primitives, and the tensor maps of the standard pool.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

// Byte offset of 16-byte chunk `c` (0..7) of row `r` in a 128-byte swizzled
// [rows][128 B] region.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- host side

// 5-D view of the standard pool [nb][2][bs][Hkv][d] (innermost first) with a
// 64-element x 1 head x 16 token box and 128-byte swizzle.
inline bool make_kv_map(CUtensorMap* map, const void* cache, int nb, int bs, int Hkv, int d) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(bs), 2, static_cast<cuuint64_t>(nb)};
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t strides[4] = {row, row * Hkv, row * Hkv * bs, row * Hkv * bs * 2};
  const cuuint32_t box[5] = {64, 1, 16, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The V half of the same pool viewed 5-D so that one box holds a 16-token
// piece's 64-column halves as consecutive 128-byte-swizzled [16][128 B]
// tiles: dims (innermost first) 64 columns, bs tokens, d/64 halves, Hkv
// heads, 2 nb (kv index + 2 * block); box 64 x 16 x d/64 x 1 x 1.
inline bool make_v_map(CUtensorMap* map, const void* cache, int nb, int bs, int Hkv, int d) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(d / 64),
                              static_cast<cuuint64_t>(Hkv), 2 * static_cast<cuuint64_t>(nb)};
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t strides[4] = {row * Hkv, 128, row, row * Hkv * bs};
  const cuuint32_t box[5] = {64, 16, static_cast<cuuint32_t>(d / 64), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace pa
