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
// warp takes a token: its rows pass in steps of 32 / (d / 8) rows, d/8 lanes to
// a row, eight values to a lane.  A lane holds both halves of its pairs (values
// 4l.. and r/2 + 4l.., two 8-byte loads), so the rotation needs no exchange
// between lanes and the sum of squares is the only reduction; weight times
// cosine and sine is formed once per token and kept in registers over its
// rows; arithmetic is on packed pairs of fp32.  18432 tokens of 32 / 8 heads,
// d 128 (457 MB): 72.5 us, 6.3 TB/s, 0.93 of the copy rate.  Before: a CTA per
// token, 16-byte loads and the other half by shuffles 207 us, a warp per token
// 131 us (instructions); one loop over all kinds of rows with loads a round
// ahead 98 us (spilled registers).  An e4m3 pool adds a division per
// value: 8191 tokens of 64 / 8 heads, d 64 (160 MB): 34.4 us.
#include <type_traits>

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
  unsigned num_tokens, shares;
  int per;   // warps per token above, steps per warp here
};

// Pairs of fp32 in one 64-bit register (fma.rn.f32x2 and the like: each half
// rounded as its scalar counterpart).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 swap2(F2 a) {
  const float2 f = split(a);
  return f2(f.y, f.x);
}
// Two bf16 (low half first) as fp32.
__device__ __forceinline__ F2 widen(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(F2 a) {
  const float2 f = split(a);
  return pack_bf16(f.x, f.y);
}

// x / scale, correctly rounded, by a multiplication and one correction
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990: with r the rounded reciprocal and q near x / s, q + r (x -
// q s), the remainder exact by fma, rounds to the quotient).  Magnitudes from
// 480 on saturate and those below 2^-20 become a zero of their sign, whatever
// their last bits (infinities, NaN and -0 among them); scales outside [2^-100,
// 2^100], whose reciprocal could leave the normal range, take the division.
__device__ __forceinline__ float quotient(float x, float scale, float r, bool plain) {
  if (!plain) return __fdiv_rn(x, scale);
  const float q = x * r;
  const uint32_t above = (__float_as_uint(q) & 0x7fffffffu) - __float_as_uint(0x1p-20f);
  return above < __float_as_uint(480.f) - __float_as_uint(0x1p-20f)
             ? fmaf(fmaf(-q, scale, x), r, q) : q;
}

// Four values as e4m3 codes of value / scale (IEEE quotient, saturating).
__device__ __forceinline__ uint32_t quant4(F2 a, F2 b, float scale, float r, bool plain) {
  const float2 x = split(a), y = split(b);
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(quotient(x.x, scale, r, plain), quotient(x.y, scale, r, plain)), __NV_SATFINITE,
      __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(quotient(y.x, scale, r, plain), quotient(y.y, scale, r, plain)), __NV_SATFINITE,
      __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

constexpr int kWarps = 4;    // units per CTA
constexpr int kFlight = 4;   // steps whose loads are in flight per warp

enum Kind { kQuery, kKey, kValue };

template <int D, bool FP8>
__global__ void __launch_bounds__(kWarps * 32, 8) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int L = D / 8;              // lanes per row
  constexpr int G = 32 / L;             // rows per step
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, l = lane % L, g = lane / L;
  // Unit = (token, share of its steps); steps run over the queries, then the
  // keys, then the values, G rows each (the last of a kind may be partial).
  const unsigned unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const unsigned t = unit / a.shares;
  if (t >= a.num_tokens) return;   // whole warps
  const int share = static_cast<int>(unit - t * a.shares);
  // The lane's two chunks of four values: the halves of four pairs where they
  // are rotated, neighbours otherwise.
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  const bool apart = !a.interleaved && turned;
  const int c0 = apart ? l : 2 * l, c1 = apart ? l + half / 4 : 2 * l + 1;

  // Where this token's keys and values go (null: nowhere), and its angles.
  const int64_t slot = a.slots[t];
  const float* angles = nullptr;
  if (a.rot > 0) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_position) {
      if (lane == 0 && share == 0) record_error(a.err, PA_DEVERR_POSITION);
      return;
    }
    angles = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
  }
  const bool keep = slot >= 0 && slot < a.num_slots;
  if (slot >= a.num_slots && lane == 0 && share == 0) record_error(a.err, PA_DEVERR_SLOT);
  constexpr int kEl = FP8 ? 1 : 2;
  uint8_t* cell = static_cast<uint8_t*>(a.cache);   // the token's keys in its block
  if (keep) {
    const int64_t blk = a.bs_log2 >= 0 ? slot >> a.bs_log2 : slot / a.bs;
    const int off = static_cast<int>(slot - blk * a.bs);
    cell += (blk * 2 * a.bs + off) * a.Hkv * (D * kEl);
  }
  const bool norm = a.q_weight != nullptr;

  // All rows of one kind that lie in this unit's share.
  int s0 = share * a.per, s1 = s0 + a.per;   // steps left, counted from the kind's first
  auto rows = [&](auto kind_tag, const __nv_bfloat16* src, int H, const __nv_bfloat16* weight) {
    constexpr Kind kind = decltype(kind_tag)::value;
    const int steps = (H + G - 1) / G;
    const int end = min(s1, steps);
    // y = rstd (A own + B other): A = w cos, B = -+ w_other sin; [chunk][pair].
    F2 A[2][2], B[2][2];
    if (kind != kValue && s0 < end) {
      F2 w[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        w[k][0] = w[k][1] = f2(1.f, 1.f);
        if (norm) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(weight + 4 * (k ? c1 : c0)));
          w[k][0] = widen(x.x);
          w[k][1] = widen(x.y);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) A[k][e] = w[k][e];
      }
      if (turned) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(angles + 4 * l));
        const float4 s = __ldg(reinterpret_cast<const float4*>(angles + half + 4 * l));
        if (apart) {
          const F2 cc[2] = {f2(c.x, c.y), f2(c.z, c.w)};
          const F2 sp[2] = {f2(s.x, s.y), f2(s.z, s.w)};
          const F2 sn[2] = {f2(-s.x, -s.y), f2(-s.z, -s.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            B[0][e] = mul2(w[1][e], sn[e]);
            B[1][e] = mul2(w[0][e], sp[e]);
            A[0][e] = mul2(w[0][e], cc[e]);
            A[1][e] = mul2(w[1][e], cc[e]);
          }
        } else {   // pairs 4l .. 4l + 3, inside the lane
          const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              B[k][e] = mul2(swap2(w[k][e]), f2(-s4[2 * k + e], s4[2 * k + e]));
              A[k][e] = mul2(w[k][e], f2(c4[2 * k + e], c4[2 * k + e]));
            }
        }
      }
    }
    const float scale = kind == kValue ? a.v_scale : a.k_scale, inv = __frcp_rn(scale);
    const bool plain = scale >= 0x1p-100f && scale <= 0x1p100f;
    uint8_t* dst = kind == kQuery
                       ? reinterpret_cast<uint8_t*>(a.q_out + static_cast<int64_t>(t) * a.Hq * D)
                       : cell + (kind == kValue ? static_cast<int64_t>(a.bs) * a.Hkv : 0) * (D * kEl);
    for (int base = s0; base < end; base += kFlight) {
      uint2 raw[kFlight][2];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r = (base + u) * G + g;
        raw[u][0] = raw[u][1] = make_uint2(0, 0);
        if (base + u < end && r < H) {
          const uint2* p = reinterpret_cast<const uint2*>(src + r * D);
          raw[u][0] = __ldcs(p + c0);
          raw[u][1] = __ldcs(p + c1);
        }
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        if (base + u >= end) break;
        const int r = (base + u) * G + g;
        const bool store = r < H && (kind == kQuery || keep);
        const uint2 x0 = raw[u][0], x1 = raw[u][1];
        if (kind == kValue && !FP8) {   // a bit copy
          if (store) {
            uint2* p = reinterpret_cast<uint2*>(dst + r * (D * 2));
            p[c0] = x0;
            p[c1] = x1;
          }
          continue;
        }
        F2 y[2][2] = {{widen(x0.x), widen(x0.y)}, {widen(x1.x), widen(x1.y)}};
        if (kind != kValue) {
          float rstd = 1.f;
          if (norm) {
            F2 s2 = mul2(y[0][0], y[0][0]);
            s2 = fma2(y[0][1], y[0][1], s2);
            s2 = fma2(y[1][0], y[1][0], s2);
            s2 = fma2(y[1][1], y[1][1], s2);
            const float2 f = split(s2);
            float ss = f.x + f.y;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rstd = rsqrtf(ss * (1.f / D) + a.eps);
          }
          F2 z[2][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            z[0][e] = y[0][e];
            z[1][e] = y[1][e];
            y[0][e] = mul2(y[0][e], A[0][e]);
            y[1][e] = mul2(y[1][e], A[1][e]);
          }
          if (apart) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[0][e] = fma2(z[1][e], B[0][e], y[0][e]);
              y[1][e] = fma2(z[0][e], B[1][e], y[1][e]);
            }
          } else if (turned) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[0][e] = fma2(swap2(z[0][e]), B[0][e], y[0][e]);
              y[1][e] = fma2(swap2(z[1][e]), B[1][e], y[1][e]);
            }
          }
          if (norm) {
            const F2 r2 = f2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[0][e] = mul2(y[0][e], r2);
              y[1][e] = mul2(y[1][e], r2);
            }
          }
        }
        if (!store) continue;
        if (kind != kQuery && FP8) {
          uint32_t* p = reinterpret_cast<uint32_t*>(dst + r * D);
          p[c0] = quant4(y[0][0], y[0][1], scale, inv, plain);
          p[c1] = quant4(y[1][0], y[1][1], scale, inv, plain);
        } else {
          uint2* p = reinterpret_cast<uint2*>(dst + r * (D * 2));
          p[c0] = make_uint2(narrow(y[0][0]), narrow(y[0][1]));
          p[c1] = make_uint2(narrow(y[1][0]), narrow(y[1][1]));
        }
      }
    }
    s0 = max(s0 - steps, 0);
    s1 = max(s1 - steps, 0);
  };
  rows(std::integral_constant<Kind, kQuery>(), a.q + t * a.q_stride, a.Hq, a.q_weight);
  rows(std::integral_constant<Kind, kKey>(), a.k + t * a.k_stride, a.Hkv, a.k_weight);
  rows(std::integral_constant<Kind, kValue>(), a.v + t * a.v_stride, a.Hkv, nullptr);
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
  // One warp per token; a batch of few tokens deals each token's steps out
  // over several warps, until about 16 warps per SM have work.
  const int rows = 32 / (n.d / 8);
  const int steps = (n.Hq + rows - 1) / rows + 2 * ((n.Hkv + rows - 1) / rows);
  long long shares = (16LL * n.sm_count + n.num_tokens - 1) / n.num_tokens;
  if (shares > steps) shares = steps;
  a.per = static_cast<int>((steps + shares - 1) / shares);
  a.shares = (steps + a.per - 1) / a.per;
  a.num_tokens = n.num_tokens;
  // shares > 1 only below 16 tokens per SM: the units fit 32 bits.
  const unsigned units = static_cast<unsigned>(n.num_tokens) * a.shares;
  const dim3 grid((units + kWarps - 1) / kWarps), block(kWarps * 32);
  if (n.d == 128)
    return n.fp8 ? launch_pdl(norm_rope_kernel<128, true>, grid, block, 0, stream, a)
                 : launch_pdl(norm_rope_kernel<128, false>, grid, block, 0, stream, a);
  return n.fp8 ? launch_pdl(norm_rope_kernel<64, true>, grid, block, 0, stream, a)
               : launch_pdl(norm_rope_kernel<64, false>, grid, block, 0, stream, a);
}

}  // namespace pa
