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
// 4l.. and r/2 + 4l.., two 8-byte loads; neighbouring pairs come in one of 16),
// so the rotation needs no exchange between lanes and the sum of squares is the
// only reduction; weight times cosine and sine is formed once per token and
// kept in registers over its rows; arithmetic is on packed pairs of fp32.
// 18432 tokens of 32 / 8 heads, d 128 (457 MB): 70.2 us, 6.5 TB/s, 0.96 of the
// copy rate; 64 tokens 2.3 us (an empty kernel 2.2).  Before: a CTA per
// token, 16-byte loads and the other half by shuffles 207 us, a warp per token
// 131 us (instructions); one loop over all kinds of rows with loads a round
// ahead 98 us (spilled registers).  An e4m3 pool adds a quotient
// per value: 8191 tokens of 64 / 8 heads, d 64, neighbouring pairs (161 MB): 30.1
// us, 0.79 of the copy rate (issue slots 53 % busy).
// Between a few tokens per SM and several waves of warps (32 per SM: 4864 tokens
// on 152 SMs) the last, part-filled wave costs most: 32 / 8 heads, d 128, bf16 /
// e4m3, times the floor of their bytes: 2048 tokens 10.7 / 11.4 us (1.41 / 1.63),
// 2500 14.6 / 17.1 (1.58 / 2.01), 4096 18.3 / 19.3 (1.21 / 1.39), 5000 26.4 / 27.5
// (1.43 / 1.62), 8191 33.7 / 34.8 (1.11 / 1.25), 18432 70.3 / 72.3 (1.04 / 1.17).
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
// Two bf16 (low half first) as fp32.
__device__ __forceinline__ F2 widen(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(F2 a) {
  const float2 f = split(a);
  return pack_bf16(f.x, f.y);
}

// min(max(x, -lim), lim); NaN stays.
__device__ __forceinline__ float clamped(float x, float lim) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(lim));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-lim));
  return x;
}
__device__ __forceinline__ float signed_as(float y, float x) {
  return __uint_as_float((__float_as_uint(y) & 0x7fffffffu) | (__float_as_uint(x) & 0x80000000u));
}

// x / scale, correctly rounded, by a multiplication and one correction
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990: with r the rounded reciprocal and q near x / s, q + r (x -
// q s), the remainder exact by fma, rounds to the quotient).  Quotients from
// 480 on saturate whatever they are, so x is held to 480 s, which keeps
// infinities out of the remainder; those below 2^-20 become a zero whatever
// their last bits, whose sign (and that of -0) is put back.  Scales outside
// [2^-100, 2^100], whose reciprocal could leave the normal range, take the
// division.  In pairs: 18432 tokens of 32 / 8 heads, d 128, 72.3 us; one value
// at a time, with the range tested instead, 2 us more.
__device__ __forceinline__ float2 quotient(F2 x, float scale, float r, bool plain) {
  float2 f = split(x);
  if (!plain) return make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
  const float lim = 480.f * scale;
  f.x = clamped(f.x, lim), f.y = clamped(f.y, lim);
  const F2 c = f2(f.x, f.y), q = mul2(c, f2(r, r));
  const float2 y = split(fma2(fma2(q, f2(-scale, -scale), c), f2(r, r), q));
  return make_float2(signed_as(y.x, f.x), signed_as(y.y, f.y));
}

// Four values as e4m3 codes of value / scale (IEEE quotient, saturating).
__device__ __forceinline__ uint32_t quant4(F2 a, F2 b, float scale, float r, bool plain) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(quotient(a, scale, r, plain), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(quotient(b, scale, r, plain), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

constexpr int kWarps = 4;    // units per CTA
constexpr int kFlight = 4;   // steps whose loads are in flight per warp

enum Kind { kQuery, kKey, kValue };

// Eight values of a lane as two vectors of four, P and Q, whose elements are
// the pairs to be rotated: two chunks of a row half a rotation apart, or (INTER)
// the even and the odd elements of 16 bytes.
struct Pairs {
  F2 p[2], q[2];
};
template <bool INTER>
__device__ __forceinline__ Pairs widen8(uint4 x) {
  if (!INTER) return {{widen(x.x), widen(x.y)}, {widen(x.z), widen(x.w)}};
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  return {{f2(lo(x.x), lo(x.y)), f2(lo(x.z), lo(x.w))},
          {f2(hi(x.x), hi(x.y)), f2(hi(x.z), hi(x.w))}};
}
// The eight values in the row's order again, as pairs of neighbours.
template <bool INTER>
__device__ __forceinline__ void in_order(const Pairs& y, F2 (&v)[4]) {
  if constexpr (!INTER) {
    v[0] = y.p[0], v[1] = y.p[1], v[2] = y.q[0], v[3] = y.q[1];
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 a = split(y.p[e]), b = split(y.q[e]);
      v[2 * e] = f2(a.x, b.x);
      v[2 * e + 1] = f2(a.y, b.y);
    }
  }
}

template <int D, bool FP8, bool INTER>
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
  // are rotated and lie apart, neighbours otherwise.
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  const int c0 = !INTER && turned ? l : 2 * l, c1 = !INTER && turned ? l + half / 4 : 2 * l + 1;
  // Rows are read once, past L1 (18432 tokens, d 128, 70.2 us, 8191 tokens, d 64,
  // e4m3 pool, 30.1; with loads that mark their lines as first to go 71.0 and 30.9).
  auto fetch = [&](const __nv_bfloat16* row, bool once) -> uint4 {
    if (INTER) {
      const uint4* p = reinterpret_cast<const uint4*>(row) + l;
      return once ? __ldcg(p) : __ldg(p);
    }
    const uint2* p = reinterpret_cast<const uint2*>(row);
    const uint2 x = once ? __ldcg(p + c0) : __ldg(p + c0);
    const uint2 y = once ? __ldcg(p + c1) : __ldg(p + c1);
    return make_uint4(x.x, x.y, y.x, y.y);
  };

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
    constexpr int kOutEl = kind == kQuery ? 2 : kEl;
    const int steps = (H + G - 1) / G;
    const int end = min(s1, steps);
    const int mine = min(end, (H - g + G - 1) / G);   // this lane's rows end here
    // y = rstd (A own + B other): A = w cos, B = -+ w_other sin.
    F2 Ap[2], Aq[2], Bp[2], Bq[2];
    if (kind != kValue && s0 < end) {
      Pairs w = {{f2(1.f, 1.f), f2(1.f, 1.f)}, {f2(1.f, 1.f), f2(1.f, 1.f)}};
      if (norm) w = widen8<INTER>(fetch(weight, false));
#pragma unroll
      for (int e = 0; e < 2; ++e) Ap[e] = w.p[e], Aq[e] = w.q[e];
      if (turned) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(angles + 4 * l));
        const float4 s = __ldg(reinterpret_cast<const float4*>(angles + half + 4 * l));
        const F2 cc[2] = {f2(c.x, c.y), f2(c.z, c.w)};
        const F2 sp[2] = {f2(s.x, s.y), f2(s.z, s.w)};
        const F2 sn[2] = {f2(-s.x, -s.y), f2(-s.z, -s.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          Bp[e] = mul2(w.q[e], sn[e]);
          Bq[e] = mul2(w.p[e], sp[e]);
          Ap[e] = mul2(w.p[e], cc[e]);
          Aq[e] = mul2(w.q[e], cc[e]);
        }
      }
    }
    uint8_t* dst = cell;
    if (kind == kQuery)
      dst = reinterpret_cast<uint8_t*>(a.q_out + static_cast<int64_t>(t) * a.Hq * D);
    else if (kind == kValue)
      dst += static_cast<int64_t>(a.bs) * a.Hkv * (D * kEl);
    const float scale = kind == kValue ? a.v_scale : a.k_scale, inv = __frcp_rn(scale);
    const bool plain = scale >= 0x1p-100f && scale <= 0x1p100f;
    for (int base = s0; base < end; base += kFlight) {
      const __nv_bfloat16* in = src + (base * G + g) * D;
      uint8_t* to = dst + (base * G + g) * (D * kOutEl);
      uint4 raw[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        raw[u] = base + u < mine ? fetch(in + u * G * D, true) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        if (base + u >= end) break;
        const bool store = base + u < mine && (kind == kQuery || keep);
        const uint4 x = raw[u];
        uint2* out = reinterpret_cast<uint2*>(to + u * (G * D * kOutEl));
        if (kind == kValue && !FP8) {   // a bit copy
          if (store) {
            if (INTER) {
              reinterpret_cast<uint4*>(out)[l] = x;
            } else {
              out[c0] = make_uint2(x.x, x.y);
              out[c1] = make_uint2(x.z, x.w);
            }
          }
          continue;
        }
        Pairs y = widen8<INTER>(x);
        if (kind != kValue) {
          float rstd = 1.f;
          if (norm) {
            F2 s2 = mul2(y.p[0], y.p[0]);
            s2 = fma2(y.p[1], y.p[1], s2);
            s2 = fma2(y.q[0], y.q[0], s2);
            s2 = fma2(y.q[1], y.q[1], s2);
            const float2 f = split(s2);
            float ss = f.x + f.y;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rstd = rsqrtf(ss * (1.f / D) + a.eps);
          }
          const Pairs z = y;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            y.p[e] = mul2(y.p[e], Ap[e]);
            y.q[e] = mul2(y.q[e], Aq[e]);
          }
          if (turned) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y.p[e] = fma2(z.q[e], Bp[e], y.p[e]);
              y.q[e] = fma2(z.p[e], Bq[e], y.q[e]);
            }
          }
          if (norm) {
            const F2 r2 = f2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y.p[e] = mul2(y.p[e], r2);
              y.q[e] = mul2(y.q[e], r2);
            }
          }
        }
        if (!store) continue;
        F2 v[4];
        in_order<INTER>(y, v);
        if (kind != kQuery && FP8) {
          const uint2 codes = make_uint2(quant4(v[0], v[1], scale, inv, plain),
                                         quant4(v[2], v[3], scale, inv, plain));
          if (INTER) {
            out[l] = codes;
          } else {
            reinterpret_cast<uint32_t*>(out)[c0] = codes.x;
            reinterpret_cast<uint32_t*>(out)[c1] = codes.y;
          }
        } else if (INTER) {
          reinterpret_cast<uint4*>(out)[l] =
              make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
        } else {
          out[c0] = make_uint2(narrow(v[0]), narrow(v[1]));
          out[c1] = make_uint2(narrow(v[2]), narrow(v[3]));
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

template <int D, bool FP8>
cudaError_t launch_t(const NormRopeArgs& a, unsigned ctas, cudaStream_t stream) {
  return a.interleaved ? launch_pdl(norm_rope_kernel<D, FP8, true>, dim3(ctas), dim3(kWarps * 32),
                                    0, stream, a)
                       : launch_pdl(norm_rope_kernel<D, FP8, false>, dim3(ctas), dim3(kWarps * 32),
                                    0, stream, a);
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
  const unsigned ctas = (units + kWarps - 1) / kWarps;
  if (n.d == 128) return n.fp8 ? launch_t<128, true>(a, ctas, stream)
                               : launch_t<128, false>(a, ctas, stream);
  return n.fp8 ? launch_t<64, true>(a, ctas, stream) : launch_t<64, false>(a, ctas, stream);
}

}  // namespace pa
