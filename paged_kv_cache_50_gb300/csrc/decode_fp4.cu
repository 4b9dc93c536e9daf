// Decode attention over a 4-bit pool (layout: fp4.cuh), stage 1 of two, or alone
// where the context is not split: o = softmax(scale q K^T) V for one query per
// request, with K, V = code * scale * k_scale (v_scale).
//
// One CTA serves one (split, kv head, request): a producer warp fetches the
// split's tokens, 16 at a time (keys, values and their scales are one run of 18 d
// bytes: one bulk copy), into a ring of stages of 32 tokens for each of eight
// consumer warps.  A consumer warp takes its 32 tokens of a stage as two M = 16
// tiles of mma.m16n8k16 with the group's query heads as N (8 per n-tile): S^T = K
// Q^T, one online softmax step over the 32 tokens (two thirds of the shuffles of
// two steps over 16), O^T += V^T P^T.  Codes are widened to f16 and multiplied by
// their scales on the way into operand registers (exact); q and the weights are f16.
//
// Bound by issue slots beside HBM: 2304 bytes for 16 tokens (d = 128) pass in 100
// cycles of an SM, in which it issues 400 warp instructions, and a sub-block needs 64
// conversions, 64 scalings and 16 MMAs before anything else.
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

namespace {

constexpr int kConsumers = 8;                      // warps
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kPieces = 2;                         // 16-token pieces of a warp in a stage

struct Fp4Args {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int max_blocks, Hq, Hkv, grp, bs, bs_log2, num_blocks;
  int S, chunk;       // splits, tokens per split (a multiple of 16)
  int positions;      // of a table row, at most INT_MAX - 1023
  float scale_log2;   // scale * k_scale * log2(e)
  float out_scale;    // v_scale
  float* ws;          // [N, Hq, S, d + 1], unused where S == 1 and no logits
  float* logits;      // [N, Hkv, logit_tokens, grp] (log2 units), or null
  int logit_tokens;
  __nv_bfloat16* out; // S == 1
  float* lse;
  int* err;
};

template <int D, int NT>
struct Fp4Cfg {
  static constexpr int kPairBytes = 2 * fp4::tile_bytes(D);
  static constexpr int kStageBytes = kConsumers * kPieces * kPairBytes;
  // Two CTAs per SM.
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kHeads = 8 * NT;
  // Rows of the merge buffer: places d + d / 16, an odd number of words apart for
  // the eight dims that a warp's lanes store at once.
  static constexpr int kOStride = D == 128 ? 164 : 68;
  static constexpr int kMergeBytes = kConsumers * kHeads * (kOStride + 2) * 4;
  static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kOffBar = kDataBytes;              // full[stage], empty[stage]
  static constexpr int kOffValid = kOffBar + 16 * kStages;   // pieces loaded, a word per stage
  static constexpr int kSmemBytes = kOffValid + 4 * kStages + 128;
  __device__ static __forceinline__ int place(int dim) { return dim + (dim >> 4); }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t q_pair(const __nv_bfloat16* p) {
  const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  return pack_f16(f.x, f.y);
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a));
}

template <int D, int NT, bool LOGITS>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) decode_fp4_kernel(const __grid_constant__ Fp4Args a) {
  using C = Fp4Cfg<D, NT>;
  constexpr int kK = D / 16;          // k-steps of K Q^T = d-tiles of V^T P^T
  constexpr int kWk = D / 32;         // words of a key row in a lane: D / 4 codes
  constexpr int kWv = D / 64;         // words of a value row in a lane: D / 8 codes
  constexpr float kRescale = 8.f;     // log2 units
  extern __shared__ __align__(128) uint8_t smem[];
  const int s = blockIdx.x, kvh = blockIdx.y, i = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;
  const int grp = a.grp;
  const uint32_t base = smem_u32(smem);
  auto full = [&](int st) { return base + C::kOffBar + 16 * st; };
  auto empty = [&](int st) { return base + C::kOffBar + 16 * st + 8; };
  volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + C::kOffValid);

  if (threadIdx.x == 0) {
#pragma unroll
    for (int st = 0; st < C::kStages; ++st) {
      tc::mbar_init(full(st), 1);
      tc::mbar_init(empty(st), kConsumers);
    }
    tc::fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  const int seq = max(0, a.seq_lens[i]);
  const int end = min(seq, a.positions);   // what lies past the table's columns has no block
  if (end < seq && s == 0 && threadIdx.x == 0) record_error(a.err, PA_DEVERR_BLOCK_ID);
  const long long a0 = static_cast<long long>(s) * a.chunk;
  const int t0 = static_cast<int>(a0 < end ? a0 : end);
  const int t1 = static_cast<int>(s == a.S - 1 || a0 + a.chunk > end ? end : a0 + a.chunk);
  const int pieces = (t1 - t0 + 15) >> 4;
  const int stages = (pieces + kConsumers * kPieces - 1) / (kConsumers * kPieces);
  const int64_t row0 = static_cast<int64_t>(i) * a.Hq + kvh * grp;
  if (pieces == 0 && a.S > 1) {
    pdl_trigger();
    for (int idx = threadIdx.x; idx < grp * (D + 1); idx += kThreads) {
      const int r = idx / (D + 1), e = idx - r * (D + 1);
      a.ws[((row0 + r) * a.S + s) * (D + 1) + e] = e == D ? -CUDART_INF_F : 0.f;
    }
    return;
  }

  float m_r[NT][2], l_r[NT][2], o[NT][kK][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_r[nt][0] = m_r[nt][1] = -CUDART_INF_F;
    l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
    for (int md = 0; md < kK; ++md)
      o[nt][md][0] = o[nt][md][1] = o[nt][md][2] = o[nt][md][3] = 0.f;
  }

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    // Lane l: piece l of a stage (of kConsumers * kPieces); warp w's are w *
    // kPieces, ....  Block ids are read a stage ahead.
    const int32_t* table = a.block_table + static_cast<int64_t>(i) * a.max_blocks;
    const bool box = lane < kConsumers * kPieces;
    auto lookup = [&](int st) {
      const int p = st * (kConsumers * kPieces) + lane;
      // (A plain load: the table may be the previous kernel's output.)
      return box && p < pieces ? table[div_bs(t0 + 16 * p, a.bs, a.bs_log2)] : -1;
    };
    int blk = lookup(0);
    for (int st = 0; st < stages; ++st) {
      const int next = st + 1 < stages ? lookup(st + 1) : -1;
      const int at = st % C::kStages, use = st / C::kStages;
      if (use > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(empty(at), (use - 1) & 1))) {
        if (lane == 0) record_error(a.err, PA_DEVERR_TIMEOUT);
        break;
      }
      const int p = st * (kConsumers * kPieces) + lane;
      const bool mine = box && p < pieces;
      const bool good = mine && blk >= 0 && blk < a.num_blocks;
      const unsigned loaded = __ballot_sync(0xffffffffu, good);
      const unsigned bad = __ballot_sync(0xffffffffu, mine && !good);
      if (lane == 0) {
        if (bad != 0u) record_error(a.err, PA_DEVERR_BLOCK_ID);
        valid[at] = loaded;
        tc::mbar_arrive_expect_tx(full(at), __popc(loaded) * C::kPairBytes);
      }
      __syncwarp();
      if (good) {
        const int tok = t0 + 16 * p;
        const int g = mod_bs(tok, a.bs, a.bs_log2) >> 4;
        bulk_load(base + at * C::kStageBytes + lane * C::kPairBytes,
                  a.cache + fp4::pair_at(blk, kvh, g, a.Hkv, a.bs >> 4, D), C::kPairBytes, full(at));
      }
      blk = next;
    }
  } else {
    // ------------------------------------------------------------ consumers
    uint32_t qf[NT][kK][2];
    {
      const __nv_bfloat16* qb = a.q + row0 * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + gid;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
          qf[nt][kk][0] = qf[nt][kk][1] = 0u;
          if (h < grp) {
            const __nv_bfloat16* p = qb + h * D + tid4 * (D / 4) + kk * 4;
            qf[nt][kk][0] = q_pair(p);
            qf[nt][kk][1] = q_pair(p + 2);
          }
        }
      }
    }
    // Source lanes of the P^T operand (tokens 2 tid4 and 2 tid4 + 1 of head gid).
    const int src_a = 8 * tid4 + (gid >> 1), src_b = src_a + 4;
    const uint32_t sel = (gid & 1) ? 0x7632u : 0x5410u;
    bool ok = true;
    for (int st = 0; st < stages; ++st) {
      const int at = st % C::kStages;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(full(at), (st / C::kStages) & 1))) {
        ok = false;
        break;
      }
      const int p0 = st * (kConsumers * kPieces) + warp * kPieces;
      const uint32_t here = valid[at] >> (warp * kPieces);
      // Visible tokens of each piece.
      int lim[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        lim[p] = (here >> p) & 1u ? min(16, t1 - (t0 + 16 * (p0 + p))) : 0;
      // (Logits are written for every token, also where a block is missing.)
      if (lim[0] > 0 || lim[1] > 0 || (LOGITS && p0 < pieces)) {
        const uint32_t pair = base + at * C::kStageBytes + warp * kPieces * C::kPairBytes;
        // S^T = K Q^T: rows = tokens gid, gid + 8; columns = heads.
        float x[kPieces][NT][4];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const uint32_t kb = pair + p * C::kPairBytes, ks = kb + 8 * D;
          uint32_t k0[kWk], k1[kWk], s0[kK / 4], s1[kK / 4];
          lds_words(kb + gid * (D / 2) + tid4 * (D / 8), k0);
          lds_words(kb + (gid + 8) * (D / 2) + tid4 * (D / 8), k1);
          if constexpr (D == 128) {
            const uint32_t c0 = fp4::widen_scales(lds_u16(ks + gid * 8 + tid4 * 2));
            const uint32_t c1 = fp4::widen_scales(lds_u16(ks + (gid + 8) * 8 + tid4 * 2));
            s0[0] = fp4::both_low(c0), s0[1] = fp4::both_high(c0);
            s1[0] = fp4::both_low(c1), s1[1] = fp4::both_high(c1);
          } else {
            s0[0] = fp4::both_low(fp4::widen_scales(lds_u8(ks + gid * 4 + tid4)));
            s1[0] = fp4::both_low(fp4::widen_scales(lds_u8(ks + (gid + 8) * 4 + tid4)));
          }
          float s2[NT][2][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              s2[nt][h][0] = s2[nt][h][1] = s2[nt][h][2] = s2[nt][h][3] = 0.f;
#pragma unroll
          for (int w = 0; w < kWk; ++w) {
            uint32_t f0[4], f1[4];
            fp4::widen8(k0[w], f0);
            fp4::widen8(k1[w], f1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t am[4] = {
                  fp4::mul2(f0[2 * h], s0[w / 2]), fp4::mul2(f1[2 * h], s1[w / 2]),
                  fp4::mul2(f0[2 * h + 1], s0[w / 2]), fp4::mul2(f1[2 * h + 1], s1[w / 2])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(s2[nt][h], am, qf[nt][2 * w + h][0], qf[nt][2 * w + h][1]);
            }
          }
          const bool v0 = gid < lim[p], v1 = gid + 8 < lim[p];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[p][nt][e] = (e < 2 ? v0 : v1) ? (s2[nt][0][e] + s2[nt][1][e]) * a.scale_log2
                                              : -CUDART_INF_F;
          if constexpr (LOGITS) {
            const int tok = t0 + 16 * (p0 + p) + gid;
            float* dst = a.logits + ((static_cast<int64_t>(i) * a.Hkv + kvh) * a.logit_tokens + tok) * grp;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int h = nt * 8 + 2 * tid4 + (e & 1);
                if (h < grp && tok + 8 * (e >> 1) < min(t1, a.logit_tokens))
                  dst[8 * (e >> 1) * grp + h] = x[p][nt][e];
              }
          }
        }
        // Online softmax in the log2 domain; the reference maximum moves only when
        // the 32 tokens' exceeds it by more than kRescale, so that weights stay < 2^8.
        uint32_t pb[kPieces][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[kPieces][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(fmaxf(x[0][nt][j], x[0][nt][2 + j]), fmaxf(x[1][nt][j], x[1][nt][2 + j]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (mx > m_r[nt][j] + kRescale) {
              const float alpha = fast_exp2(m_r[nt][j] - mx);   // 0 when the old one is -inf
              m_r[nt][j] = mx;
              l_r[nt][j] *= alpha;
#pragma unroll
              for (int md = 0; md < kK; ++md) {
                o[nt][md][j] *= alpha;
                o[nt][md][2 + j] *= alpha;
              }
            }
            const float mu = m_r[nt][j] == -CUDART_INF_F ? 0.f : m_r[nt][j];
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
              pr[p][j] = fast_exp2(x[p][nt][j] - mu);
              pr[p][2 + j] = fast_exp2(x[p][nt][2 + j] - mu);
              l_r[nt][j] += pr[p][j] + pr[p][2 + j];
            }
          }
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
            const uint32_t u_lo = pack_f16(pr[p][0], pr[p][1]);   // token gid, heads 2 tid4, + 1
            const uint32_t u_hi = pack_f16(pr[p][2], pr[p][3]);   // token gid + 8
            const uint32_t xa = __shfl_sync(0xffffffffu, u_lo, src_a);
            const uint32_t xb = __shfl_sync(0xffffffffu, u_lo, src_b);
            const uint32_t ya = __shfl_sync(0xffffffffu, u_hi, src_a);
            const uint32_t yb = __shfl_sync(0xffffffffu, u_hi, src_b);
            pb[p][nt][0] = __byte_perm(xa, xb, sel);
            pb[p][nt][1] = __byte_perm(ya, yb, sel);
          }
        }
        // O^T += V^T P^T: a lane's codes are d / 8 neighbouring ones of the value rows
        // 2 tid4, + 1, + 8, + 9; two tokens' codes are interleaved by halves of bytes.
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const uint32_t vb = pair + p * C::kPairBytes + fp4::tile_bytes(D), vs = vb + 8 * D;
          uint32_t v[4][kWv], sc[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * tid4 + (r & 1) + 8 * (r >> 1);
            lds_words(vb + row * (D / 2) + gid * (D / 16), v[r]);
            sc[r] = lds_u8(vs + row * (D / 16) + (D == 128 ? gid : gid >> 1));
            // The weight of a token that is not there is 0, its codes are finite
            // whatever the bytes, but its scale need not be.
            if (row >= lim[p]) sc[r] = 0u;
          }
          const uint32_t sab = fp4::widen_scales(sc[0] | (sc[1] << 8));
          const uint32_t scd = fp4::widen_scales(sc[2] | (sc[3] << 8));
#pragma unroll
          for (int w = 0; w < kWv; ++w) {
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            uint32_t ab[2][4], cd[2][4];   // [even, odd element][word byte]
            fp4::widen8((v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), ab[0]);
            fp4::widen8(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), ab[1]);
            fp4::widen8((v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), cd[0]);
            fp4::widen8(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), cd[1]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t am[4] = {fp4::mul2(ab[0][b], sab), fp4::mul2(ab[1][b], sab),
                                      fp4::mul2(cd[0][b], scd), fp4::mul2(cd[1][b], scd)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(o[nt][4 * w + b], am, pb[p][nt][0], pb[p][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty(at));
    }
    if (!ok && lane == 0) record_error(a.err, PA_DEVERR_TIMEOUT);
  }
  pdl_trigger();

  // Every copy has landed: a stage was waited for by all consumers, or a wait has run
  // out; then the producer's last stages get one more bounded wait each.
  if (warp == kConsumers && lane == 0)
    for (int st = max(0, stages - C::kStages); st < stages; ++st)
      tc::mbar_wait(full(st % C::kStages), (st / C::kStages) & 1);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l_r[nt][j] += __shfl_xor_sync(0xffffffffu, l_r[nt][j], k);
  __syncthreads();
  float* obuf = reinterpret_cast<float*>(smem);
  float* mbuf = obuf + kConsumers * C::kHeads * C::kOStride;   // [warp][head]
  float* lbuf = mbuf + kConsumers * C::kHeads;
  if (warp < kConsumers) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int md = 0; md < kK; ++md)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = nt * 8 + 2 * tid4 + (e & 1), dim = gid * (D / 8) + 2 * md + (e >> 1);
          obuf[(warp * C::kHeads + h) * C::kOStride + C::place(dim)] = o[nt][md][e];
        }
      if (gid == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mbuf[warp * C::kHeads + nt * 8 + 2 * tid4 + j] = m_r[nt][j];
          lbuf[warp * C::kHeads + nt * 8 + 2 * tid4 + j] = l_r[nt][j];
        }
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < grp * D; idx += kThreads) {
    const int r = idx / D, e = idx % D;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, mbuf[w * C::kHeads + r]);
    float L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      const float mw = mbuf[w * C::kHeads + r];
      const float f = mw == -CUDART_INF_F ? 1.f : fast_exp2(mw - M);   // (its sums are 0, or NaN)
      L += f * lbuf[w * C::kHeads + r];
      acc += f * obuf[(w * C::kHeads + r) * C::kOStride + C::place(e)];
    }
    const float y = L == 0.f ? 0.f : acc / L * a.out_scale;
    const float ls = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
    if (a.ws == nullptr) {
      a.out[(row0 + r) * D + e] = __float2bfloat16_rn(y);
      if (e == 0 && a.lse != nullptr) a.lse[row0 + r] = ls;
    } else {
      float* dst = a.ws + ((row0 + r) * a.S + s) * (D + 1);
      dst[e] = y;
      // (A NaN row is handed on as +inf, whose weight in the merge is NaN: a maximum
      // would pass over a NaN.)
      if (e == 0) dst[D] = ls == ls ? ls : CUDART_INF_F;
    }
  }
}

template <int D, int NT, bool LOGITS>
cudaError_t launch_t(const Fp4Args& a, int N, cudaStream_t stream) {
  using C = Fp4Cfg<D, NT>;
  auto kern = decode_fp4_kernel<D, NT, LOGITS>;
  static DeviceFlags smem_set;
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.S, a.Hkv, N), dim3(kThreads), C::kSmemBytes, stream, a);
}
template <int D, int NT>
cudaError_t launch_n(const Fp4Args& a, int N, cudaStream_t stream) {
  return a.logits != nullptr ? launch_t<D, NT, true>(a, N, stream)
                             : launch_t<D, NT, false>(a, N, stream);
}

}  // namespace

// Splits of the context: about six CTAs for each SM (two are resident), of at least
// 256 tokens, so that a batch of mixed lengths evens out.
int decode_fp4_splits(int N, int Hkv, int max_seq_len, int sm_count) {
  const long long units = static_cast<long long>(N) * Hkv;
  const long long want = (6LL * sm_count + units - 1) / std::max(1LL, units);
  const long long most = (static_cast<long long>(max_seq_len) + 255) / 256;
  return static_cast<int>(std::max(1LL, std::min({want, most, 64LL})));
}

cudaError_t launch_decode_fp4(const DecodeFp4Launch& n, cudaStream_t stream) {
  Fp4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(n.q);
  a.cache = static_cast<const uint8_t*>(n.cache);
  a.block_table = n.block_table;
  a.seq_lens = n.seq_lens;
  a.max_blocks = n.max_blocks;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.grp = n.Hq / n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  a.num_blocks = n.num_blocks;
  a.S = n.S;
  a.chunk = static_cast<int>(split_chunk(n.max_seq_len, n.S, 16));
  a.positions = static_cast<int>(
      std::min(static_cast<long long>(n.max_blocks) * n.bs, INT_MAX - 1023LL));
  a.scale_log2 = n.scale * n.k_scale * kLog2e;
  a.out_scale = n.v_scale;
  a.ws = n.ws;
  a.logits = n.logits;
  a.logit_tokens = n.logit_tokens;
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  const bool wide = a.grp > 8;   // groups of 9 to 16 heads take two n-tiles
  if (n.d == 128) return wide ? launch_n<128, 2>(a, n.N, stream) : launch_n<128, 1>(a, n.N, stream);
  return wide ? launch_n<64, 2>(a, n.N, stream) : launch_n<64, 1>(a, n.N, stream);
}

}  // namespace pa
