// The 4-bit pool: layout, conversions, and the products of decode attention over it.
//
// A pool is [num_blocks][Hkv][bs / 16][2][9 d] bytes: for each block, kv head and
// 16 tokens a tile of keys and, behind it, one of values.  A tile is [16][d / 2]
// bytes of e2m1 codes (two a byte, the even element in the low half) and then
// [16][d / 16] e4m3 scales, one for each 16 elements of a row: element e of a row
// stands for code * scale[e / 16] * k_scale (or v_scale, the layer's).  Heads come
// before tokens and scales beside their codes, so that what attention reads for 16
// tokens of a head is one run of 18 d bytes: one bulk copy.
//
// code * scale has at most 5 significant bits and lies on a grid of 2^-10 below
// 2688: it is exact in f16, in which the tensor cores take it.
#pragma once

#include <cuda_fp4.h>

#include "pa_common.cuh"

namespace pa {
namespace fp4 {

__host__ __device__ constexpr int tile_bytes(int d) { return 9 * d; }

// Byte offset of the tile pair of tokens 16 g .. 16 g + 15 of a block.
__device__ __forceinline__ int64_t pair_at(int64_t blk, int head, int g, int Hkv, int groups, int d) {
  return ((blk * Hkv + head) * groups + g) * (2 * tile_bytes(d));
}

// Four bytes of codes -> four f16 pairs (low half: the low code).
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales (the low 16 bits) -> an f16 pair.
__device__ __forceinline__ uint32_t widen_scales(uint32_t two) {
  uint32_t h;
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %1;\ncvt.rn.f16x2.e4m3x2 %0, a;\n}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t both_low(uint32_t a) { return __byte_perm(a, a, 0x1010); }
__device__ __forceinline__ uint32_t both_high(uint32_t a) { return __byte_perm(a, a, 0x3232); }

}  // namespace fp4
}  // namespace pa
