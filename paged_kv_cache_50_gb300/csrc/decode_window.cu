// Decode attention with a sliding window and a few first tokens that stay
// visible, over a bf16 or e4m3 pool, in one launch without a workspace.
//
// Mathematics: the query at position seq - 1 sees p < sinks and p >= lo = max(0,
// seq - window); o = softmax(scale q K^T) V over those p, split over the
// tokens and merged by the partials' maxima and sums ("Chapter 1: attention
// backends", sections 3.1 and 4.1).
//
// The visible tokens form a list of 16-token sub-blocks: ceil(sinks / 16)
// first ones, then those from lo rounded down to 16 (one run from position 0
// where the two meet).  Nothing else is read.  One cluster of S CTAs serves
// one (request, kv head): CTA r takes the r-th share of the list, its four
// warps sub-blocks in turn, each warp with its own cp.async ring; the warps'
// states are merged in shared memory and the CTAs' in distributed shared
// memory, every CTA writing a share of the outputs.  A window bounds a
// request's work, so unlike split-KV decode over a whole context S <= 16
// shares are enough, and the second launch and its fp32 workspace (written
// and read once) go.
//
// Bound by HBM where the batch fills the GPU, else by latency (lengths ->
// block ids -> K/V -> merge, one after the other).
#include <algorithm>
#include <climits>

#include "decode_core.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

namespace {

struct WindowArgs {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int max_blocks, Hq, Hkv, bs, bs_log2, num_blocks;
  float scale_log2;   // scale * k_scale * log2(e)
  float out_scale;    // v_scale
  int window, sinks;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

template <class KV, int D, int STAGES, int NT>
struct WindowCfg {
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStageBytes = 2 * KV::kTileBytes;   // K + V
  static constexpr int kWarpBytes = STAGES * kStageBytes;
  static constexpr int kPipeBytes = kWarps * kWarpBytes;
  static constexpr int kHeads = 8 * NT;
  // Combine buffer: O rows per warp, then max, sum and divisor per (warp,
  // head), then the CTA's max, sum and divisor per head.
  static constexpr int kCombineBytes = (kWarps * kHeads * (KV::kOStride + 3) + 3 * kHeads) * 4;
  static constexpr int kSmemBytes = kPipeBytes > kCombineBytes ? kPipeBytes : kCombineBytes;
};

__device__ __forceinline__ float ld_remote(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <class KV, int D, int STAGES, int NT>
__global__ void __launch_bounds__(128) decode_window_kernel(const WindowArgs a) {
  using C = WindowCfg<KV, D, STAGES, NT>;
  constexpr int kK = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int S = gridDim.x, s = blockIdx.x, kvh = blockIdx.y, i = blockIdx.z;   // cluster = grid.x
  const int grp = a.Hq / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;

  pdl_wait();
  const int seq = min(max(0, a.seq_lens[i]), INT_MAX - 64);   // sums below stay in range
  const int32_t* table = a.block_table + static_cast<int64_t>(i) * a.max_blocks;
  const int lo = seq > a.window ? seq - a.window : 0;
  const int sinks = min(a.sinks, seq);
  int n_first = (sinks + 15) >> 4, wb = lo & ~15;
  if (wb <= 16 * n_first) n_first = wb = 0;   // the first tokens reach the window: one run
  // 16-token sub-blocks of the list, and this CTA's share [v0, v1) of them.
  const int nsb = n_first + static_cast<int>((static_cast<unsigned>(seq - wb) + 15u) >> 4);
  const int per = (nsb + S - 1) / S;
  const int v_begin = min(nsb, s * per), v_end = min(nsb, v_begin + per);
  const int my_n = v_end - v_begin > warp ? (v_end - v_begin - warp + C::kWarps - 1) / C::kWarps : 0;
  // First position of the warp's n-th sub-block.
  auto token = [&](int n) {
    const int v = v_begin + warp + n * C::kWarps;
    return v < n_first ? 16 * v : wb + 16 * (v - n_first);
  };
  auto visible = [&](int p) { return p < seq && (p >= lo || p < sinks); };
  auto lookup = [&](int n) {
    return block_at(table, div_bs(token(n), a.bs, a.bs_log2), a.max_blocks);
  };
  int first_blk[STAGES];
#pragma unroll
  for (int n = 0; n < STAGES; ++n) first_blk[n] = n < my_n ? lookup(n) : -1;

  uint32_t qf[NT][kK][2];
  {
    const __nv_bfloat16* qb =
        a.q + (static_cast<int64_t>(i) * a.Hq + static_cast<int64_t>(kvh) * grp) * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gid;
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        qf[nt][kk][0] = qf[nt][kk][1] = 0u;
        if (h < grp) KV::load_q(qb + h * D, tid4, kk, qf[nt][kk]);
      }
    }
  }

  const uint32_t wbase = smem_u32(smem) + warp * C::kWarpBytes;
  const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * KV::kRowBytes;
  // Bit n % 32: the n-th sub-block's block id was valid.
  uint32_t okbits = 0;
  auto issue = [&](int n, int blk) {
    const int tb = token(n);
    const bool ok = blk >= 0 && blk < a.num_blocks;
    if (!ok && lane == 0) record_error(a.err, PA_DEVERR_BLOCK_ID);
    okbits = (okbits & ~(1u << (n & 31))) | (static_cast<uint32_t>(ok) << (n & 31));
    const int off = mod_bs(tb, a.bs, a.bs_log2);
    const uint8_t* kbase = a.cache +
                           (static_cast<int64_t>(ok ? blk : 0) * 2 * a.bs + off) * row_bytes +
                           static_cast<int64_t>(kvh) * KV::kRowBytes;
    const uint8_t* vbase = kbase + a.bs * row_bytes;
    const uint32_t kdst = wbase + (n % STAGES) * C::kStageBytes;
    const uint32_t vdst = kdst + KV::kTileBytes;
#pragma unroll
    for (int k = 0; k < 16 * KV::kChunks / 32; ++k) {
      const int c = lane + 32 * k;
      const int r = c / KV::kChunks, cc = c % KV::kChunks;
      const int bytes = ok && visible(tb + r) ? 16 : 0;   // others: zeros, nothing read
      const uint32_t so = KV::at(r, cc);
      cp_async_16(kdst + so, kbase + r * row_bytes + cc * 16, bytes);
      cp_async_16(vdst + so, vbase + r * row_bytes + cc * 16, bytes);
    }
  };

  dec::State<D, NT> st;
  st.clear();
#pragma unroll
  for (int n = 0; n < STAGES - 1; ++n) {
    if (n < my_n) issue(n, first_blk[n]);
    cp_async_commit();
  }
  int next_blk = STAGES - 1 < my_n ? first_blk[STAGES - 1] : -1;
  for (int n = 0; n < my_n; ++n) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    if (n + STAGES - 1 < my_n) {
      issue(n + STAGES - 1, next_blk);
      if (n + STAGES < my_n) next_blk = lookup(n + STAGES);
    }
    cp_async_commit();
    const int tb = token(n);
    const bool ok = (okbits >> (n & 31)) & 1u;
    const uint32_t kb = wbase + (n % STAGES) * C::kStageBytes;
    dec::add_sub_block<KV, D, NT>(st, kb, kb + KV::kTileBytes, lane, ok && visible(tb + gid),
                                  ok && visible(tb + gid + 8), a.scale_log2, qf);
  }
  cp_async_wait<0>();
  pdl_trigger();

  // Sums over the 8 token lanes.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.l[nt][j] += __shfl_xor_sync(0xffffffffu, st.l[nt][j], o);
        if (KV::kRoundedSums) st.lr[nt][j] += __shfl_xor_sync(0xffffffffu, st.lr[nt][j], o);
      }

  // The four warps' states -> this CTA's (max, sum, divisor, O) per head, in
  // place of warp 0's O rows.
  __syncthreads();
  float* obuf = reinterpret_cast<float*>(smem);
  float* mbuf = obuf + C::kWarps * C::kHeads * KV::kOStride;   // [warp][head]
  float* lbuf = mbuf + C::kWarps * C::kHeads;
  float* rbuf = lbuf + C::kWarps * C::kHeads;
  float* cta = rbuf + C::kWarps * C::kHeads;                   // [3][head]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int md = 0; md < kK; ++md)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = nt * 8 + 2 * tid4 + (e & 1);
        obuf[(warp * C::kHeads + h) * KV::kOStride + KV::place(KV::dim(md, e, gid))] =
            st.o[nt][md][e];
      }
    if (gid == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = warp * C::kHeads + nt * 8 + 2 * tid4 + j;
        mbuf[at] = st.m[nt][j];
        lbuf[at] = st.l[nt][j];
        rbuf[at] = KV::kRoundedSums ? st.lr[nt][j] : st.l[nt][j];
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < grp * D; idx += C::kThreads) {
    const int r = idx / D, e = idx % D;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, mbuf[w * C::kHeads + r]);
    float L = 0.f, LR = 0.f, acc = 0.f;
    if (M != -CUDART_INF_F) {
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float f = fast_exp2(mbuf[w * C::kHeads + r] - M);
        L += f * lbuf[w * C::kHeads + r];
        LR += f * rbuf[w * C::kHeads + r];
        acc += f * obuf[(w * C::kHeads + r) * KV::kOStride + KV::place(e)];
      }
    }
    const int64_t row = static_cast<int64_t>(i) * a.Hq + kvh * grp + r;
    if (S == 1) {
      a.out[row * D + e] = __float2bfloat16_rn(LR == 0.f ? 0.f : acc / LR * a.out_scale);
      if (e == 0 && a.lse != nullptr)
        a.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
    } else {
      obuf[r * KV::kOStride + KV::place(e)] = acc;   // only this thread reads it
      if (e == 0) {
        cta[r] = M;
        cta[C::kHeads + r] = L;
        cta[2 * C::kHeads + r] = LR;
      }
    }
  }
  if (S == 1) return;
  tc::cluster_sync();
  // Merge over the cluster: the outputs are dealt out over its CTAs.
  const uint32_t o_at = smem_u32(obuf), c_at = smem_u32(cta);
  for (int idx = s * C::kThreads + threadIdx.x; idx < grp * D; idx += S * C::kThreads) {
    const int r = idx / D, e = idx % D;
    const uint32_t oa = o_at + (r * KV::kOStride + KV::place(e)) * 4, ca = c_at + r * 4;
    float m[16], M = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      m[k] = k < S ? ld_remote(tc::map_to_rank(ca, k)) : -CUDART_INF_F;
      M = fmaxf(M, m[k]);
    }
    float L = 0.f, LR = 0.f, acc = 0.f;
    if (M != -CUDART_INF_F) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k < S) {
          const float f = fast_exp2(m[k] - M);
          L += f * ld_remote(tc::map_to_rank(ca + C::kHeads * 4, k));
          LR += f * ld_remote(tc::map_to_rank(ca + 2 * C::kHeads * 4, k));
          acc += f * ld_remote(tc::map_to_rank(oa, k));
        }
      }
    }
    const int64_t row = static_cast<int64_t>(i) * a.Hq + kvh * grp + r;
    a.out[row * D + e] = __float2bfloat16_rn(LR == 0.f ? 0.f : acc / LR * a.out_scale);
    if (e == 0 && a.lse != nullptr)
      a.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
  }
  tc::cluster_sync();   // no CTA leaves while another reads its shared memory
}

template <class KV, int D, int STAGES, int NT>
cudaError_t launch_t(const DecodeWindowLaunch& n, const WindowArgs& a, int S, cudaStream_t stream) {
  using C = WindowCfg<KV, D, STAGES, NT>;
  auto kern = decode_window_kernel<KV, D, STAGES, NT>;
  static DeviceFlags smem_set, cluster_set;
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  if (S > 8) {
    // Clusters of more than 8 CTAs are opt-in.
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev >= 64 || !cluster_set.done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) cluster_set.done[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, n.Hkv, n.N);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

// CTAs per (request, kv head): enough for about 12 CTAs per SM, as the
// split-KV planner, at least 16 sub-blocks (4 per warp) each, a power of two
// up to 16.
int decode_window_shares(int N, int Hkv, long long visible, int sm_count) {
  const long long units = static_cast<long long>(N) * Hkv;
  const long long want = (12LL * sm_count + units - 1) / units;
  const long long most = visible / 256;
  int S = 1;
  while (S < 16 && S < want && 2 * S <= most) S *= 2;
  return S;
}

cudaError_t launch_decode_window(const DecodeWindowLaunch& n, cudaStream_t stream) {
  WindowArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(n.q);
  a.cache = static_cast<const uint8_t*>(n.cache);
  a.block_table = n.block_table;
  a.seq_lens = n.seq_lens;
  a.max_blocks = n.max_blocks;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  a.num_blocks = n.num_blocks;
  a.scale_log2 = n.scale * n.k_scale * kLog2e;
  a.out_scale = n.v_scale;
  a.window = n.window;
  a.sinks = n.sinks;
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  const long long table = static_cast<long long>(n.max_blocks) * n.bs;
  const long long visible = std::min(static_cast<long long>(n.window) + n.sinks, table);
  const int S = decode_window_shares(n.N, n.Hkv, visible, n.sm_count);
  const bool wide = n.Hq / n.Hkv > 8;   // groups of 9..16 heads take two n-tiles
  using dec::KvBf16;
  using dec::KvE4m3;
  if (n.fp8) {
    if (n.d == 128)
      return wide ? launch_t<KvE4m3<128>, 128, 4, 2>(n, a, S, stream)
                  : launch_t<KvE4m3<128>, 128, 3, 1>(n, a, S, stream);
    return wide ? launch_t<KvE4m3<64>, 64, 8, 2>(n, a, S, stream)
                : launch_t<KvE4m3<64>, 64, 8, 1>(n, a, S, stream);
  }
  if (n.d == 128)
    return wide ? launch_t<KvBf16<128>, 128, 2, 2>(n, a, S, stream)
                : launch_t<KvBf16<128>, 128, 2, 1>(n, a, S, stream);
  return wide ? launch_t<KvBf16<64>, 64, 4, 2>(n, a, S, stream)
              : launch_t<KvBf16<64>, 64, 4, 1>(n, a, S, stream);
}

}  // namespace pa
