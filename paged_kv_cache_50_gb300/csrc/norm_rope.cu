// Norms of queries and keys for each head, the position rotation and the
// cache write (step 1 of the paged-kernel contract, "Attention Backends",
// section "What 'paged attention' requires of a kernel") in one pass over the
// projection's output.
//
// Mathematics, in fp32 with one rounding at the end: y = x w / sqrt(mean(x^2)
// + eps) over a head's d values, then (a, b) -> (a cos - b sin, b cos + a sin)
// over the pairs of the first r values.  The cosines and sines come from a
// table (fp32, computed once in fp64): position * frequency in fp32 would be
// off by 2^-25 * 131072 radians at far positions.
//
// Bound by HBM: every input is read once and every output written once.  A
// group of d/8 lanes holds one head row, 16 bytes a lane, so that a row is one
// coalesced load and one store; the sum of squares is a shuffle reduction
// inside the group.  The halves of a pair k, k + r/2 sit r/16 lanes apart:
// the raw bf16 words are exchanged (4 shuffles instead of 8 for the fp32
// values) and both lanes scale them alike.  A lane's place in its row is the
// same for every row it takes, so weights, cosines and sines stay in
// registers over a token's rows, and the loads of up to kRows rows are in
// flight together with the position -> table chain.
#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

struct NormRopeArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  const __nv_bfloat16* q_weight;   // both weights or none
  const __nv_bfloat16* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  void* cache;
  __nv_bfloat16* q_out;
  int* err;
  int64_t num_slots;
  float eps, k_scale, v_scale;
  int max_position, rot, interleaved, Hq, Hkv, bs, bs_log2;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// Eight values as e4m3 codes of value / scale (IEEE quotient, saturating).
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float scale) {
  uint32_t r[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = make_float2(__fdiv_rn(f[2 * k], scale), __fdiv_rn(f[2 * k + 1], scale));
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    r[k >> 1] |= static_cast<uint32_t>(c) << (16 * (k & 1));
  }
  return make_uint2(r[0], r[1]);
}

constexpr int kThreads = 256;
constexpr int kRows = 3;   // rows of a token in flight per group

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int L = D / 8;              // lanes per row
  constexpr int G = kThreads / L;       // rows in flight per CTA and step
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  const int rows = a.Hq + 2 * a.Hkv;
  const int step = G * gridDim.y;
  const int first = blockIdx.y * G + g;

  const uint4* qsrc = reinterpret_cast<const uint4*>(a.q + t * a.q_stride) + l;
  const uint4* ksrc = reinterpret_cast<const uint4*>(a.k + t * a.k_stride) + l;
  const uint4* vsrc = reinterpret_cast<const uint4*>(a.v + t * a.v_stride) + l;
  auto load = [&](int r) -> uint4 {
    if (r < a.Hq) return __ldcs(qsrc + r * L);
    if (r < a.Hq + a.Hkv) return __ldcs(ksrc + (r - a.Hq) * L);
    if (r < rows) return __ldcs(vsrc + (r - a.Hq - a.Hkv) * L);
    return make_uint4(0, 0, 0, 0);
  };
  uint4 raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) raw[u] = load(first + u * step);

  // Where this token's keys and values go (< 0: nowhere).
  int64_t slot = a.slots[t];
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(a.err, PA_DEVERR_SLOT);
    slot = -1;
  }
  // This lane's weights, its rotation and its pair's lane.  c, s: cos and
  // signed sin for the eight values, y_own c + y_pair s.
  const bool norm = a.q_weight != nullptr;
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq, wqp = wq, wkp = wq;
  float c[8], s[8];
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  int pair = l;
  if (a.rot > 0) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_position) {
      if (threadIdx.x == 0 && blockIdx.y == 0) record_error(a.err, PA_DEVERR_POSITION);
      return;
    }
    if (turned) {
      const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
      if (a.interleaved) {
        // Pairs 4l .. 4l + 3 inside the lane: (c, -s), (c, s).
        const float4 cc = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
        const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
        const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c[2 * k] = c[2 * k + 1] = c4[k];
          s[2 * k] = -s4[k];
          s[2 * k + 1] = s4[k];
        }
      } else {
        const bool low = 8 * l < half;
        pair = low ? l + half / 8 : l - half / 8;
        const int k0 = low ? 8 * l : 8 * l - half;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 cc = __ldg(reinterpret_cast<const float4*>(row + k0) + k);
          const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + k0) + k);
          c[4 * k] = cc.x, c[4 * k + 1] = cc.y, c[4 * k + 2] = cc.z, c[4 * k + 3] = cc.w;
          s[4 * k] = ss.x, s[4 * k + 1] = ss.y, s[4 * k + 2] = ss.z, s[4 * k + 3] = ss.w;
        }
        if (low) {
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] = -s[k];
        }
      }
    }
  }
  if (norm) {
    wq = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + l);
    wk = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + l);
    wqp = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + pair);
    wkp = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + pair);
  }
  const int lane = threadIdx.x & 31;
  const int src_lane = (lane & ~(L - 1)) | pair;
  const int64_t blk = slot < 0 ? 0 : (a.bs_log2 >= 0 ? slot >> a.bs_log2 : slot / a.bs);
  const int off = slot < 0 ? 0 : static_cast<int>(slot - blk * a.bs);

  // Whole warps only: the groups of a warp differ in r by less than a warp's
  // rows, and rows past the end take part in the shuffles with zeros.
  for (int base = first; base - g < rows; base += kRows * step) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = base + u * step;
      if (r - g >= rows) break;   // uniform over the CTA
      const uint4 x = raw[u];
      raw[u] = load(r + kRows * step);
      const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
      float y[8];
      unpack8(x, y);
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(y[k], y[k], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      uint4 xp;
      xp.x = __shfl_sync(0xffffffffu, x.x, src_lane);
      xp.y = __shfl_sync(0xffffffffu, x.y, src_lane);
      xp.z = __shfl_sync(0xffffffffu, x.z, src_lane);
      xp.w = __shfl_sync(0xffffffffu, x.w, src_lane);
      if (!is_v) {
        const float rstd = norm ? rsqrtf(ss * (1.f / D) + a.eps) : 1.f;
        if (norm) {
          float w[8];
          unpack8(is_q ? wq : wk, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = y[k] * rstd * w[k];
        }
        if (turned) {
          float z[8];
          if (a.interleaved) {
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] = y[k ^ 1];
          } else {
            unpack8(xp, z);
            if (norm) {
              float w[8];
              unpack8(is_q ? wqp : wkp, w);
#pragma unroll
              for (int k = 0; k < 8; ++k) z[k] = z[k] * rstd * w[k];
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = fmaf(y[k], c[k], z[k] * s[k]);
        }
      }
      if (is_q) {
        reinterpret_cast<uint4*>(a.q_out)[(t * a.Hq + r) * L + l] = pack8(y);
      } else if (slot >= 0 && r < rows) {
        const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
        const int64_t row = ((blk * 2 + (is_v ? 1 : 0)) * a.bs + off) * a.Hkv + h;
        if (FP8)
          static_cast<uint2*>(a.cache)[row * L + l] = quant8(y, is_v ? a.v_scale : a.k_scale);
        else
          static_cast<uint4*>(a.cache)[row * L + l] = is_v ? x : pack8(y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& n, cudaStream_t stream) {
  NormRopeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(n.q);
  a.k = static_cast<const __nv_bfloat16*>(n.key);
  a.v = static_cast<const __nv_bfloat16*>(n.value);
  a.q_stride = n.q_stride;
  a.k_stride = n.key_stride;
  a.v_stride = n.value_stride;
  a.q_weight = static_cast<const __nv_bfloat16*>(n.q_weight);
  a.k_weight = static_cast<const __nv_bfloat16*>(n.k_weight);
  a.cos_sin = n.cos_sin;
  a.positions = n.positions;
  a.slots = n.slot_mapping;
  a.cache = n.cache;
  a.q_out = static_cast<__nv_bfloat16*>(n.q_out);
  a.err = n.err;
  a.num_slots = static_cast<int64_t>(n.num_blocks) * n.bs;
  a.eps = n.eps;
  a.k_scale = n.k_scale;
  a.v_scale = n.v_scale;
  a.max_position = n.max_position;
  a.rot = n.rotary_dim;
  a.interleaved = n.interleaved;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  // One CTA per token; a batch of few tokens spreads each token's rows over
  // several, up to two CTAs per SM.
  const int groups = kThreads / (n.d / 8);
  const int by_rows = (n.Hq + 2 * n.Hkv + groups - 1) / groups;
  int split = (2 * n.sm_count + n.num_tokens - 1) / n.num_tokens;
  if (split > by_rows) split = by_rows;
  const dim3 grid(n.num_tokens, split);
  if (n.d == 128)
    return n.fp8 ? launch_pdl(norm_rope_kernel<128, true>, grid, dim3(kThreads), 0, stream, a)
                 : launch_pdl(norm_rope_kernel<128, false>, grid, dim3(kThreads), 0, stream, a);
  return n.fp8 ? launch_pdl(norm_rope_kernel<64, true>, grid, dim3(kThreads), 0, stream, a)
               : launch_pdl(norm_rope_kernel<64, false>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace pa
