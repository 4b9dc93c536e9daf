// One 16-token sub-block of decode attention for the query heads of one kv
// group, by one warp: the products and the online softmax of the windowed
// decode kernel, for a bf16 pool and for a pool of e4m3 codes.  (The split-KV
// kernels of decode.cu and decode_fp8.cu hold their own, over tiles that
// cp.async lays out: a change here does not reach them.)
//
// The 16 tokens are the M dimension of mma.m16n8k16 and the group's heads its
// N dimension (8 per n-tile): S^T = K Q^T, softmax over the tokens (two in a
// lane, the rest across the 8 lanes that share tid4), O^T += V^T P^T.  The
// reference max moves only when a sub-block's max exceeds it by more than 8
// (log2 units), so rescaling O is rare and weights stay below 2^8.
#pragma once

#include <math_constants.h>

#include "pa_common.cuh"

namespace pa {
namespace dec {

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Four e4m3 codes (byte 0 lowest) -> two f16x2 words, exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// bf16 pool: operands as they are, read by ldmatrix; the weights are rounded
// to bf16 for the PV product, and the output's divisor sums the rounded ones.
template <int D>
struct KvBf16 {
  static constexpr int kChunks = D / 8;          // 16-byte chunks per token row
  static constexpr int kTileBytes = 16 * D * 2;  // 16 tokens of K or V
  static constexpr int kGroups = D / 64;         // 128-byte column groups of a row
  static constexpr bool kRoundedSums = true;
  // Combine buffer row: = 4 mod 32 floats apart, no bank conflict.
  static constexpr int kOStride = D + 4;
  // Byte offset of chunk c of token row r: [d / 64][16 tokens][128 B],
  // 128-byte swizzled, as the TMA box of a tile lays it out.
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * 2048 + r * 128 + (((c ^ r) & 7) << 4));
  }
  __device__ static __forceinline__ void load_q(const __nv_bfloat16* row, int tid4, int kk,
                                                uint32_t (&f)[2]) {
    f[0] = *reinterpret_cast<const uint32_t*>(row + kk * 16 + 2 * tid4);
    f[1] = *reinterpret_cast<const uint32_t*>(row + kk * 16 + 8 + 2 * tid4);
  }
  template <int NT>
  __device__ static __forceinline__ void scores(uint32_t kb, int lane,
                                                const uint32_t (&qf)[NT][D / 16][2],
                                                float (&s2)[NT][2][4]) {
    const int row = lane & 15, half = lane >> 4;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      ldmatrix_x4(kb + at(row, 2 * kk + half), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_bf16_16816(s2[nt][kk & 1], a, qf[nt][kk][0], qf[nt][kk][1]);
    }
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16(lo, hi); }
  template <int NT>
  __device__ static __forceinline__ void values(uint32_t vb, int lane, const uint32_t (&pb)[NT][2],
                                                float (&o)[NT][D / 16][4]) {
    const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
    for (int md = 0; md < D / 16; ++md) {
      uint32_t a[4];
      ldmatrix_x4_trans(vb + at(row, 2 * md + half), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[nt][md], a, pb[nt][0], pb[nt][1]);
    }
  }
  // Head dimension of accumulator (md, e) in a lane, and its place in a
  // combine row.
  __device__ static __forceinline__ int dim(int md, int e, int gid) {
    return md * 16 + gid + 8 * (e >> 1);
  }
  __device__ static __forceinline__ int place(int dim) { return dim; }
};

// e4m3 pool: codes widen to f16 exactly on their way into operand registers,
// q is rounded to f16, weights are packed as f16.  The head dimension is
// permuted alike in K and Q (a lane's words of a row are contiguous), and V's
// rows so that a lane's codes are d/8 contiguous ones.
template <int D>
struct KvE4m3 {
  static constexpr int kChunks = D / 16;
  static constexpr int kTileBytes = 16 * D;
  static constexpr int kGroups = 1;
  static constexpr bool kRoundedSums = false;
  static constexpr int kOStride = D == 128 ? 164 : 68;
  // [16 tokens][d B], swizzled over 128 (d = 128) or 64 bytes.
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    if constexpr (D == 128)
      return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
    else
      return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  __device__ static __forceinline__ uint32_t q_pair(const __nv_bfloat16* p) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
    return pack_f16(f.x, f.y);
  }
  __device__ static __forceinline__ void load_q(const __nv_bfloat16* row, int tid4, int kk,
                                                uint32_t (&f)[2]) {
    const int c0 = tid4 * (D / 4) + kk * 4;
    f[0] = q_pair(row + c0);
    f[1] = q_pair(row + c0 + 2);
  }
  template <int WORDS>
  __device__ static __forceinline__ void row_words(uint32_t tile, int r, int byte0,
                                                   uint32_t (&w)[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
      for (int k = 0; k < WORDS / 4; ++k) {
        const uint4 x = lds128(tile + at(r, byte0 / 16 + k));
        w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
      }
    } else {
      static_assert(WORDS == 2, "8-byte rows only");
      const uint2 x = lds64(tile + at(r, byte0 / 16) + (byte0 & 8));
      w[0] = x.x, w[1] = x.y;
    }
  }
  template <int NT>
  __device__ static __forceinline__ void scores(uint32_t kb, int lane,
                                                const uint32_t (&qf)[NT][D / 16][2],
                                                float (&s2)[NT][2][4]) {
    const int gid = lane >> 2, tid4 = lane & 3;
    uint32_t k0[D / 16], k1[D / 16];
    row_words<D / 16>(kb, gid, tid4 * (D / 4), k0);
    row_words<D / 16>(kb, gid + 8, tid4 * (D / 4), k1);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      e4m3x4_to_f16(k0[kk], a[0], a[2]);
      e4m3x4_to_f16(k1[kk], a[1], a[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_f16_16816(s2[nt][kk & 1], a, qf[nt][kk][0], qf[nt][kk][1]);
    }
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16(lo, hi); }
  template <int NT>
  __device__ static __forceinline__ void values(uint32_t vb, int lane, const uint32_t (&pb)[NT][2],
                                                float (&o)[NT][D / 16][4]) {
    constexpr int kW = D / 32;
    const int gid = lane >> 2, tid4 = lane & 3;
    uint32_t va[kW], vb1[kW], vc[kW], ve[kW];
    const int ra = 2 * tid4, byte0 = gid * (D / 8);
    row_words<kW>(vb, ra, byte0, va);
    row_words<kW>(vb, ra + 1, byte0, vb1);
    row_words<kW>(vb, ra + 8, byte0, vc);
    row_words<kW>(vb, ra + 9, byte0, ve);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t c01[4], c89[4];
      e4m3x4_to_f16(__byte_perm(va[w], vb1[w], 0x5140), c01[0], c01[1]);
      e4m3x4_to_f16(__byte_perm(va[w], vb1[w], 0x7362), c01[2], c01[3]);
      e4m3x4_to_f16(__byte_perm(vc[w], ve[w], 0x5140), c89[0], c89[1]);
      e4m3x4_to_f16(__byte_perm(vc[w], ve[w], 0x7362), c89[2], c89[3]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {c01[2 * h], c01[2 * h + 1], c89[2 * h], c89[2 * h + 1]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][2 * w + h], a, pb[nt][0], pb[nt][1]);
      }
    }
  }
  __device__ static __forceinline__ int dim(int md, int e, int gid) {
    return gid * (D / 8) + 2 * md + (e >> 1);
  }
  __device__ static __forceinline__ int place(int dim) { return dim + (dim >> 4); }
};

// A warp's running state: per lane the heads nt * 8 + 2 tid4 + {0, 1}.
template <int D, int NT>
struct State {
  float m[NT][2];    // reference max (log2 units), alike over the token lanes
  float l[NT][2];    // sum of the weights of this lane's tokens
  float lr[NT][2];   // sum of the rounded weights (kRoundedSums)
  float o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = lr[nt][0] = lr[nt][1] = 0.f;
#pragma unroll
      for (int md = 0; md < D / 16; ++md)
        o[nt][md][0] = o[nt][md][1] = o[nt][md][2] = o[nt][md][3] = 0.f;
    }
  }
};

// The softmax weights of a sub-block (as the PV product's operand pb) from its
// K tile at kb in shared memory, with the state's maxima and sums moved on;
// v0, v1: whether this lane's tokens gid and gid + 8 are visible (rows that
// are not hold zeros).  KV::values adds the sub-block's V tile afterwards.
template <class KV, int D, int NT>
__device__ __forceinline__ void weights(State<D, NT>& st, uint32_t kb, int lane, bool v0, bool v1,
                                        float scale_log2, const uint32_t (&qf)[NT][D / 16][2],
                                        uint32_t (&pb)[NT][2]) {
  constexpr float kRescale = 8.f;
  const int gid = lane >> 2, tid4 = lane & 3;
  // Even and odd k-steps in two chains of half the length.
  float s2[NT][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) s2[nt][h][0] = s2[nt][h][1] = s2[nt][h][2] = s2[nt][h][3] = 0.f;
  KV::template scores<NT>(kb, lane, qf, s2);
  // Source lanes of the P^T operand: tokens 2 tid4 (a) and 2 tid4 + 1 (b) of
  // head gid are in the lane of tid4' = gid / 2, half gid % 2.
  const int src_a = 8 * tid4 + (gid >> 1), src_b = src_a + 4;
  const uint32_t sel = (gid & 1) ? 0x7632u : 0x5410u;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float p[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float x0 = v0 ? (s2[nt][0][j] + s2[nt][1][j]) * scale_log2 : -CUDART_INF_F;
      const float x1 = v1 ? (s2[nt][0][2 + j] + s2[nt][1][2 + j]) * scale_log2 : -CUDART_INF_F;
      float mx = fmaxf(x0, x1);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      if (mx > st.m[nt][j] + kRescale) {
        const float alpha = fast_exp2(st.m[nt][j] - mx);   // 0 when the old max is -inf
        st.m[nt][j] = mx;
        st.l[nt][j] *= alpha;
        if (KV::kRoundedSums) st.lr[nt][j] *= alpha;
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          st.o[nt][md][j] *= alpha;
          st.o[nt][md][2 + j] *= alpha;
        }
      }
      const float mu = st.m[nt][j] == -CUDART_INF_F ? 0.f : st.m[nt][j];
      p[j] = fast_exp2(x0 - mu);
      p[2 + j] = fast_exp2(x1 - mu);
      st.l[nt][j] += p[j] + p[2 + j];
    }
    const uint32_t u_lo = KV::pack(p[0], p[1]);   // token gid, heads 2 tid4, + 1
    const uint32_t u_hi = KV::pack(p[2], p[3]);   // token gid + 8
    if (KV::kRoundedSums) {
      add_bf16x2_f32(st.lr[nt][0], st.lr[nt][1], u_lo);
      add_bf16x2_f32(st.lr[nt][0], st.lr[nt][1], u_hi);
    }
    const uint32_t xa = __shfl_sync(0xffffffffu, u_lo, src_a);
    const uint32_t xb = __shfl_sync(0xffffffffu, u_lo, src_b);
    const uint32_t ya = __shfl_sync(0xffffffffu, u_hi, src_a);
    const uint32_t yb = __shfl_sync(0xffffffffu, u_hi, src_b);
    pb[nt][0] = __byte_perm(xa, xb, sel);
    pb[nt][1] = __byte_perm(ya, yb, sel);
  }
}

}  // namespace dec
}  // namespace pa
