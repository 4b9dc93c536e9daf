// Decode's second stage with the weights' sums: the merge of what the first left
// (split partials, as merge.cu takes them, or the states of decode_fp4.cu's cut units),
// and for each cached token p of request i and kv head h
//   scores[i][h][p] += sum over the group's heads g of exp(x_g[p] - lse_g),
// x the logits that stage 1 left beside its partials.
//
// Stage 1 cannot add the weights itself: a token's weight needs the row's whole
// sum.  What it leaves is 4 bytes for each token and query head, against 144 (4-bit
// pool) or 512 (bf16) of keys and values for each token and kv head; for most
// batches they are still in L2 when this kernel reads them.  A token's sum is
// formed by one thread in the order of the heads: no atomics, the same result every
// time.
//
// The first CTAs of a (request, kv head) merge the outputs, the others take 2048 tokens
// each.  Every CTA finds the group's log-sum-exps itself from the splits' (at most a
// few hundred floats, in L2), with the logits of its tokens on their way meanwhile.
//
// Bound by the logits' bytes and the CTAs' starts: 128 requests of up to 8192 tokens,
// 32 heads (75 MB of logits, 38 MB of sums) 26 us, 1024 tokens each 28, 4096 each 30.
#include <math_constants.h>

#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 2048;   // of a CTA
constexpr int kMaxGroup = 16;
constexpr int kFewStates = 16;
constexpr int kFewUnits = 64;

struct ScoreArgs {
  const float* ws;
  const float* parts;
  const int2* spans;
  const float* row_lse;
  float out_scale;
  int positions;
  const float* logits;
  const int32_t* seq_lens;
  float* scores;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  int S, Hq, Hkv, grp, max_seq_len;
  int merging;        // CTAs of a (request, kv head) that merge, before those that add
  int64_t logit_tokens, score_tokens;
};

// 2^x for a weight: below 2^-126 it adds nothing to a sum, and is 0.
__device__ __forceinline__ float small_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// VW: floats of a token's logits per load.
template <int D, int VW>
__global__ void __launch_bounds__(kScoreThreads) decode_scores_kernel(
    const __grid_constant__ ScoreArgs a) {
  // Per row: the states' maximum, their sum, and the log-sum-exp.
  __shared__ __align__(16) float row_m[kMaxGroup], row_l[kMaxGroup], row_x[kMaxGroup];
  __shared__ float factor[kScoreThreads], partial[kScoreThreads];
  pdl_wait();
  pdl_trigger();
  const int kvh = blockIdx.y, i = blockIdx.z, grp = a.grp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool cut = a.spans != nullptr;
  int seq = max(0, a.seq_lens[i]);
  if (cut) seq = min(seq, a.positions);   // (what lies past them has no logits)
  // Tokens past max_seq_len have no logits.
  const int end = min(seq, a.max_seq_len);
  const bool merges = static_cast<int>(blockIdx.x) < a.merging;
  const int first = (static_cast<int>(blockIdx.x) - a.merging) * kScoreTokens;
  if (!merges && first >= end) return;
  if (blockIdx.x == 0 && threadIdx.x == 0 && end < seq) record_error(a.err, PA_DEVERR_LENGTH);
  const int64_t unit = static_cast<int64_t>(i) * a.Hkv + kvh;
  const int64_t row0 = static_cast<int64_t>(i) * a.Hq + kvh * grp;
  // State s of row r: D values, then (split partials, normalised) the log-sum-exp, or
  // (cut units, log2 units) maximum and sum.
  int states = a.S;
  int2 span = make_int2(0, 0);
  if (cut) {
    if (seq == 0) return;   // its outputs are there already
    span = a.spans[unit];
    states = span.y - span.x + 1;
  }
  auto state = [&](int r, int s) {
    return cut ? a.parts + ((static_cast<int64_t>(span.x + s) * 2 + (s == 0)) * grp + r) * (D + 2)
               : a.ws + ((row0 + r) * a.S + s) * (D + 1);
  };
  const bool done = cut && states == 1;   // ... and these
  if (done && merges) return;
  // The logits of a thread's tokens (their first VW heads) and their sums, on the way
  // while the log-sum-exps are formed.
  constexpr int kEach = kScoreTokens / kScoreThreads;
  const int tok0 = first + static_cast<int>(threadIdx.x), there = end - tok0;
  const float* x = a.logits + (unit * a.logit_tokens + tok0) * grp;
  float* sums = a.scores + unit * a.score_tokens + tok0;
  float v[kEach][VW], sum[kEach];
  auto load = [&](int g) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const float* p = x + k * kScoreThreads * grp + g;
      if (k * kScoreThreads < there) {
        if constexpr (VW == 4)
          *reinterpret_cast<float4*>(v[k]) = __ldcs(reinterpret_cast<const float4*>(p));
        else
          v[k][0] = __ldcs(p);
      }
    }
  };
  if (!merges) {
    load(0);
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (k * kScoreThreads < there) sum[k] = sums[k * kScoreThreads];
  }
  for (int r = warp; r < grp; r += kScoreThreads / 32) {
    float m = -CUDART_INF_F, l = 0.f, x;
    if (done) {
      x = a.row_lse[row0 + r];
    } else {
      for (int s = lane; s < states; s += 32) m = fmaxf(m, state(r, s)[D]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      for (int s = lane; s < states; s += 32) {
        const float* p = state(r, s);
        if (cut)
          l += (p[D] == m ? 1.f : fast_exp2(p[D] - m)) * p[D + 1];
        else
          l += p[D] == -CUDART_INF_F ? 0.f : expf(p[D] - m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      x = l == 0.f ? -CUDART_INF_F : cut ? (m + log2f(l)) * kLn2 : m + logf(l);
    }
    if (lane == 0) {
      row_m[r] = m, row_l[r] = l;
      row_x[r] = x == -CUDART_INF_F ? CUDART_INF_F : x;   // (an empty row's weights: 0)
      if (blockIdx.x == 0 && a.lse != nullptr) a.lse[row0 + r] = x;
    }
  }
  __syncthreads();
  if (merges) {
    auto factor_of = [&](float x, float m) {
      return cut ? (x == m ? 1.f : fast_exp2(x - m)) : x == -CUDART_INF_F ? 0.f : expf(x - m);
    };
    auto give = [&](int r, int e, float acc) {
      a.out[(row0 + r) * D + e] =
          __float2bfloat16_rn(row_l[r] == 0.f ? 0.f : acc / row_l[r] * a.out_scale);
    };
    const int m0 = static_cast<int>(blockIdx.x);
    if (states <= kFewStates) {
      const int rows = m0 < grp ? (grp - m0 + a.merging - 1) / a.merging : 0;
      for (int idx = threadIdx.x; idx < rows * D; idx += kScoreThreads) {
        const int r = m0 + idx / D * a.merging, e = idx % D;
        float acc = 0.f;
#pragma unroll 4
        for (int s = 0; s < states; ++s) {
          const float* p = state(r, s);
          acc += factor_of(p[D], row_m[r]) * p[e];
        }
        give(r, e, acc);
      }
      return;
    }
    // Many states: their factors once, and the states dealt over the threads of an element.
    constexpr int kParts = kScoreThreads / D;
    const int e = threadIdx.x % D, part = threadIdx.x / D;
    for (int r = m0; r < grp; r += a.merging) {
      float acc = 0.f;
      for (int s0 = 0; s0 < states; s0 += kScoreThreads) {
        const int n = min(kScoreThreads, states - s0);
        if (static_cast<int>(threadIdx.x) < n)
          factor[threadIdx.x] = factor_of(state(r, s0 + threadIdx.x)[D], row_m[r]);
        __syncthreads();
#pragma unroll 8
        for (int s = part; s < n; s += kParts) acc += factor[s] * state(r, s0 + s)[e];
        __syncthreads();
      }
      partial[threadIdx.x] = acc;
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int k = 1; k < kParts; ++k) acc += partial[threadIdx.x + k * D];
        give(r, e, acc);
      }
      __syncthreads();
    }
    return;
  }
  float w[kEach] = {};
  for (int g = 0; g < grp; g += VW) {
    if (g > 0) load(g);
    float of[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) of[e] = row_x[g + e];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
#pragma unroll
      for (int e = 0; e < VW; ++e) w[k] += small_exp2(fmaf(-kLog2e, of[e], v[k][e]));
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (k * kScoreThreads < there) sums[k * kScoreThreads] = sum[k] + w[k];
}

template <int D, int VW>
cudaError_t launch_t(const ScoreArgs& a, int N, cudaStream_t stream) {
  const long long chunks = (static_cast<long long>(a.max_seq_len) + kScoreTokens - 1) / kScoreTokens;
  return launch_pdl(decode_scores_kernel<D, VW>,
                    dim3(static_cast<unsigned>(chunks + a.merging), a.Hkv, N), dim3(kScoreThreads), 0, stream,
                    a);
}

}  // namespace

cudaError_t launch_decode_scores(const ScoresLaunch& n, cudaStream_t stream) {
  ScoreArgs a{};
  a.ws = n.ws;
  a.parts = n.parts;
  a.spans = n.spans;
  a.row_lse = n.row_lse;
  a.out_scale = n.out_scale;
  a.positions = n.positions;
  a.logits = n.logits;
  a.seq_lens = n.seq_lens;
  a.scores = n.scores;
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  a.S = n.S;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.grp = n.Hq / n.Hkv;
  a.max_seq_len = n.max_seq_len;
  a.logit_tokens = n.logit_tokens;
  a.score_tokens = n.score_tokens;
  // Few (request, kv head) pairs are cut into many parts each: a CTA for each row then.
  // (2 requests of 10210 tokens, one kv head of 16: 33 us with one for all, now 21, over a
  // 4-bit pool 103, now 36; 4 requests with 8 kv heads of 4: 37 and 36; but 16 such of 4096
  // tokens 38 and 40.)
  a.merging = static_cast<long long>(n.N) * n.Hkv < kFewUnits ? a.grp : 1;
  const bool four = a.grp % 4 == 0;
  if (n.d == 128) return four ? launch_t<128, 4>(a, n.N, stream) : launch_t<128, 1>(a, n.N, stream);
  return four ? launch_t<64, 4>(a, n.N, stream) : launch_t<64, 1>(a, n.N, stream);
}

}  // namespace pa
