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
// one (request, kv head): CTA r takes the r-th share of the list, its four,
// eight or sixteen warps sub-blocks in turn, each warp with its own ring of K and V
// tiles, filled by TMA boxes of 16 token rows of a head (a box is one instruction
// of one lane; the same ring filled by cp.async took 49.7 us instead of 42.5 on
// the batch below, its address and mask arithmetic being what a warp spent its
// time on).  The warps' states are merged in shared memory.  The CTAs send each
// other their parts of the outputs (st.async, counted on a barrier of the
// receiver), and each finishes a share of them.  A window bounds a request's
// work, so unlike split-KV decode over a whole context S <= 8 shares are enough,
// and the second launch and its fp32 workspace (written and read once) go.
//
// Bound by HBM where the batch fills the GPU, else by latency: one request of 64
// / 8 heads, window 4096, takes 8.1 us, of which the launch and the set-up are
// ~2, lengths and block ids 0.5, the first tile 0.9, two to three sub-blocks per
// warp 2.7 (a sub-block is a chain of ~1600 cycles in a warp, which is why more
// warps help), the warps' merge 0.6 and the cluster's 1.2.  Fetching the parts from the
// others between two cluster barriers instead took 1.1 us longer.  Measured (32 / 8
// heads, d 128): 64 requests, window 1024 over U[128, 4096] tokens, 242 MB: 41.0
// us, 5.9 TB/s; window 4096 over U[1024, 8192], 899 MB: 135-137 us, 6.6 TB/s; an
// e4m3 pool, 128 requests, window 4096, 911 MB: 148-151 us, 6.1 TB/s (372 warp
// instructions per 16 tokens, 64 of them conversions).
#include <algorithm>
#include <climits>

#include "decode_core.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

namespace {

struct WindowArgs {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int max_blocks, Hq, grp, bs, bs_log2, num_blocks;
  int out_share;      // outputs (heads x d) of a CTA
  int positions;      // of a table row, at most INT_MAX - 64
  float scale_log2;   // scale * k_scale * log2(e)
  float out_scale;    // v_scale
  int window, sinks;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

constexpr int kMaxShares = 8;   // the largest portable cluster

// A warp's ring has R places; while one is worked on, the next R - 1 are on
// their way.  Where a row is one column group, a place takes the K and V tiles
// of a sub-block, by one 4 KB TMA box (2 KB boxes, one for K and one for V, took
// twice as long on 64-wide bf16 rows: 87 us against 42 for 64 requests, window
// 2048); else K and V take a place and a box each.
template <class KV, int D, int R, int NT, int W>
struct WindowCfg {
  static constexpr int kWarps = W;
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kPair = KV::kGroups == 1;
  static constexpr int kPlaceBytes = (kPair ? 2 : 1) * KV::kTileBytes;
  static constexpr int kWarpBytes = R * kPlaceBytes;   // a multiple of the swizzle atom
  static constexpr int kPipeBytes = kWarps * kWarpBytes;
  static constexpr int kHeads = 8 * NT;
  // Combine buffer: O rows per warp, then max (later: factor), sum and divisor
  // per (warp, head), then the CTA's max, sum and divisor per head (16 bytes).
  static constexpr int kOffStats = kWarps * kHeads * (KV::kOStride + 3) * 4;
  static constexpr int kCombineBytes = kOffStats + kHeads * 16;
  static constexpr int kDataBytes = kPipeBytes > kCombineBytes ? kPipeBytes : kCombineBytes;
  static constexpr int kOffBar = (kDataBytes + 7) / 8 * 8;   // [warp][R] barriers
  // What the cluster's CTAs send each other, apart from the ring, which a slower
  // CTA still uses: a barrier, max, sum and divisor per (CTA, head), and a share
  // of each CTA's O.
  static constexpr int kOffReceived = (kOffBar + kWarps * R * 8 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffReceived + 1024;   // + alignment slack
  __host__ __device__ static constexpr int received_bytes(int S, int share) {
    return 16 + S * kHeads * 16 + S * share * 4;
  }
};
// Outputs of one CTA of a cluster of S, out of `total`: whole 16 bytes.
__host__ __device__ __forceinline__ int output_share(int total, int S) {
  return (total / 4 + S - 1) / S * 4;
}

// Arrival at a cluster barrier that publishes nothing but what a fence before it
// does (fence_barrier_init).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

#ifdef PA_TEST_HOOKS
// Test builds only: warp 0 of share g_decode_skip.x of the first request's
// first kv head does not issue box g_decode_skip.y; {-1, -1} = off.  With
// g_decode_late it issues it after all once the wait for it has run out.
// g_decode_left: boxes that a warp issued after a wait of its own had run out,
// and boxes that were still on their way when it had drained its ring.
__device__ int2 g_decode_skip = {-1, -1};
__device__ int g_decode_late = 0;
__device__ int2 g_decode_left = {0, 0};
__device__ __forceinline__ bool box_landed(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
#endif

template <class KV, int D, int R, int NT, int W, int MINB>
__global__ void __launch_bounds__(32 * W, MINB) decode_window_kernel(
    const __grid_constant__ CUtensorMap map, const __grid_constant__ WindowArgs a) {
  using C = WindowCfg<KV, D, R, NT, W>;
  constexpr int kAhead = C::kPair ? R - 1 : (R + 1) / 2;   // block ids in hand

  constexpr int kK = D / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int S = gridDim.x, s = blockIdx.x, kvh = blockIdx.y, i = blockIdx.z;   // cluster = grid.x
  const int grp = a.grp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;

  const uint32_t wbase = smem_u32(smem) + warp * C::kWarpBytes;
  const uint32_t bars = smem_u32(smem) + C::kOffBar + warp * R * 8;
  if (lane == 0) {
    tc::tma_prefetch_desc(&map);
#pragma unroll
    for (int k = 0; k < R; ++k) tc::mbar_init(bars + 8 * k, 1);
    if (warp == 0) tc::mbar_init(smem_u32(smem) + C::kOffReceived, 1);
    tc::fence_barrier_init();
  }
  __syncwarp();   // each warp uses its own ring's barriers only
  if (S > 1) cluster_arrive_relaxed();   // the receive barrier is set up
  pdl_wait();
  const int seq = max(0, a.seq_lens[i]);
  const int32_t* table = a.block_table + static_cast<int64_t>(i) * a.max_blocks;
  const int lo = seq > a.window ? seq - a.window : 0;
  // What lies past the table's columns has no block and is not walked over.
  const int end = min(seq, a.positions);
  if (end < seq && s == 0 && threadIdx.x == 0) record_error(a.err, PA_DEVERR_BLOCK_ID);
  const int sinks = min(a.sinks, end);
  int n_first = (sinks + 15) >> 4, wb = lo & ~15;
  if (wb <= 16 * n_first) n_first = wb = 0;   // the first tokens reach the window: one run
  // 16-token sub-blocks of the list, and this CTA's share [v0, v1) of them.
  const int nsb = n_first + ((max(0, end - wb) + 15) >> 4);
  const int per = (nsb + S - 1) / S;
  const int v_begin = min(nsb, s * per), v_end = min(nsb, v_begin + per);
  const int left = v_end - v_begin - warp;
  const int my_n = left > 0 ? (left + C::kWarps - 1) / C::kWarps : 0;
  // First position of the warp's n-th sub-block.
  auto token = [&](int n) {
    const int v = v_begin + warp + n * C::kWarps;
    return v < n_first ? 16 * v : wb + 16 * (v - n_first);
  };
  auto visible = [&](int p) { return p < end && (p >= lo || p < sinks); };
  // (A plain load: the table may be the previous kernel's output.)
  auto lookup = [&](int n) {
    const int idx = div_bs(token(n), a.bs, a.bs_log2);
    return table[idx];
  };
  // Block ids of sub-blocks n .. n + kAhead (the copies of the last one go
  // out while sub-block n is worked on).
  int ids[kAhead + 1];
#pragma unroll
  for (int n = 0; n <= kAhead; ++n) ids[n] = n < my_n ? lookup(n) : -1;

  // Box h into ring place `place`: sub-block h, or the K or V of sub-block
  // h / 2, in block blk.  A box that is not loaded (no such block) completes
  // its barrier all the same.
  int failed = -1;   // the box whose wait has run out
#ifdef PA_TEST_HOOKS
  auto hooked = [&](int h) {
    return warp == 0 && h == g_decode_skip.y && kvh == 0 && i == 0 && s == g_decode_skip.x;
  };
#endif
  auto issue = [&](int h, int blk, int place) {
    const int n = C::kPair ? h : h >> 1;
    if (lane != 0 || n >= my_n) return;
    const uint32_t bar = bars + 8 * place;
#ifdef PA_TEST_HOOKS
    if (failed < 0 && hooked(h)) return;
    if (failed >= 0 && !hooked(h)) atomicAdd(&g_decode_left.x, 1);
#endif
    if (blk >= 0 && blk < a.num_blocks) {
      const int off = mod_bs(token(n), a.bs, a.bs_log2);
      tc::mbar_arrive_expect_tx(bar, C::kPlaceBytes);
      if (C::kPair)
        tc::tma_load_5d(wbase + place * C::kPlaceBytes, &map, bar, 0, off, kvh, 0, blk);
      else
        tc::tma_load_5d(wbase + place * C::kPlaceBytes, &map, bar, 0, off, 0, kvh,
                        2 * blk + (h & 1));
    } else {
      record_error(a.err, PA_DEVERR_BLOCK_ID);
      tc::mbar_arrive(bar);
    }
  };
  int at = 0, parity = 0;   // place and barrier parity of the tile worked on
  auto arrived = [&]() {
    return __all_sync(0xffffffffu, tc::mbar_wait(bars + 8 * at, parity));
  };
  auto next_tile = [&]() {
    if (++at == R) at = 0, parity ^= 1;
  };

  // The first boxes go out before anything else that can wait for them.
#pragma unroll
  for (int h = 0; h < R - 1; ++h) issue(h, ids[C::kPair ? h : h >> 1], h);

  const int total = grp * D, out_share = a.out_share;
  const int out_begin = s * out_share, out_n = max(0, min(total - out_begin, out_share));
  const uint32_t received = smem_u32(smem) + C::kOffReceived;
  if (S > 1 && threadIdx.x == 0)
    tc::mbar_arrive_expect_tx(received, static_cast<uint32_t>(S * (out_n * 4 + grp * 16)));
  __syncwarp();
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

  dec::State<D, NT> st;
  st.clear();
  for (int n = 0; n < my_n; ++n) {
    const int blk = ids[0];
    const int after = n + kAhead + 1;   // the next block id, a sub-block ahead of its copies
    const int fetched = after < my_n ? lookup(after) : -1;
    const int tb = token(n);
    const bool ok = blk >= 0 && blk < a.num_blocks;
    // Most sub-blocks are visible as a whole.
    const bool whole = ok && tb >= lo && tb + 16 <= end;
    bool v0 = true, v1 = true;
    if (!whole) v0 = ok && visible(tb + gid), v1 = ok && visible(tb + gid + 8);
    // The next box goes to the place of the one before this.
    const int before = at == 0 ? R - 1 : at - 1;
    if (C::kPair)
      issue(n + R - 1, ids[R - 1], before);
    else
      issue(2 * n + R - 1, ids[(R - 1) >> 1], before);
    if (!arrived()) {
      failed = C::kPair ? n : 2 * n;
      break;
    }
    uint32_t pb[NT][2];
    dec::weights<KV, D, NT>(st, wbase + at * C::kPlaceBytes, lane, v0, v1, a.scale_log2, qf, pb);
    uint32_t vb = wbase + at * C::kPlaceBytes + KV::kTileBytes;
    if (!C::kPair) {
      __syncwarp();   // every lane is done with K(n): its place is free
      issue(2 * n + R, ids[R >> 1], at);
      next_tile();
      if (!arrived()) {
        failed = 2 * n + 1;
        break;
      }
      vb = wbase + at * C::kPlaceBytes;
    }
    if (__any_sync(0xffffffffu, !whole)) {
      // Weights of unseen tokens are 0, but 0 * NaN is not: clear their rows.
      for (int c = lane; c < 16 * KV::kChunks; c += 32) {
        const int r = c / KV::kChunks;
        const uint32_t dst = vb + KV::at(r, c % KV::kChunks);
        if (!(ok && visible(tb + r)))
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0u) : "memory");
      }
      tc::fence_proxy_async_smem();   // before a later TMA box lands here
      __syncwarp();
    }
    KV::template values<NT>(vb, lane, pb, st.o);
    __syncwarp();
    next_tile();
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ids[k] = ids[k + 1];
    ids[kAhead] = fetched;
  }
  if (failed >= 0 && lane == 0) {
    // Given up: the outputs are invalid.  No copy may still be landing when the
    // ring becomes the merge buffer and the CTA goes on.  The ring holds the
    // boxes failed .. failed + R - 1 (as far as there are), in this order from
    // the place that the warp stands at: each gets one more bounded wait.
    record_error(a.err, PA_DEVERR_TIMEOUT);
#ifdef PA_TEST_HOOKS
    if (hooked(failed) && g_decode_late) issue(failed, ids[0], at);
    const int at0 = at, parity0 = parity;
#endif
    const int past = min(failed + R, C::kPair ? my_n : 2 * my_n);
    for (int h = failed; h < past; ++h) {
      tc::mbar_wait(bars + 8 * at, parity);
      next_tile();
    }
#ifdef PA_TEST_HOOKS
    at = at0, parity = parity0;
    for (int h = failed; h < past; ++h) {
      if (!(hooked(h) && !g_decode_late) && !box_landed(bars + 8 * at, parity))
        atomicAdd(&g_decode_left.y, 1);
      next_tile();
    }
#endif
  }
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

  // The warps' states, in place of the ring.
  __syncthreads();
  float* obuf = reinterpret_cast<float*>(smem);
  float* mbuf = obuf + C::kWarps * C::kHeads * KV::kOStride;   // [warp][head]
  float* lbuf = mbuf + C::kWarps * C::kHeads;
  float* rbuf = lbuf + C::kWarps * C::kHeads;
  float4* stats = reinterpret_cast<float4*>(smem + C::kOffStats);   // [head]
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
  // Each warp's factor per head; a head's warps are neighbouring lanes.
  const int64_t row0 = static_cast<int64_t>(i) * a.Hq + kvh * grp;
  if (threadIdx.x < C::kWarps * C::kHeads) {   // whole warps
    const int h = threadIdx.x / C::kWarps, at = threadIdx.x % C::kWarps * C::kHeads + h;
    float M = mbuf[at];
#pragma unroll
    for (int o = 1; o < C::kWarps; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float f = M == -CUDART_INF_F ? 0.f : fast_exp2(mbuf[at] - M);
    float L = f * lbuf[at], LR = f * rbuf[at];
#pragma unroll
    for (int o = 1; o < C::kWarps; o <<= 1) {
      L += __shfl_xor_sync(0xffffffffu, L, o);
      LR += __shfl_xor_sync(0xffffffffu, LR, o);
    }
    if (S == 1) {
      f = LR == 0.f ? 0.f : f / LR * a.out_scale;
      if (threadIdx.x % C::kWarps == 0 && h < grp && a.lse != nullptr)
        a.lse[row0 + h] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
    } else if (threadIdx.x % C::kWarps == 0) {
      stats[h] = make_float4(M, L, LR, 0.f);
    }
    mbuf[at] = f;
  }
  __syncthreads();
  auto merged = [&](int idx) {
    const int r = idx / D, at = KV::place(idx % D);
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w)
      acc = fmaf(mbuf[w * C::kHeads + r], obuf[(w * C::kHeads + r) * KV::kOStride + at], acc);
    return acc;
  };
  if (S == 1) {
    for (int idx = threadIdx.x; idx < total; idx += C::kThreads)
      a.out[row0 * D + idx] = __float2bfloat16_rn(merged(idx));
    return;
  }
  // Each CTA makes a share of the outputs.  The others' parts are sent to it, not
  // fetched: one way instead of a cluster barrier and a round trip, and since
  // every CTA waits for all that is sent to it, none leaves early.
  const uint32_t stats_at = received + 16, o_at = stats_at + S * C::kHeads * 16;
  tc::cluster_wait();   // every CTA's barrier is set up
  for (int idx = 4 * threadIdx.x; idx < total; idx += 4 * C::kThreads) {
    const int owner = idx / out_share, r = idx / D, at = KV::place(idx % D);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float f = mbuf[w * C::kHeads + r];
      const float* o = obuf + (w * C::kHeads + r) * KV::kOStride + at;
      float x[4];
      if constexpr (KV::kRoundedSums) {
        const float4 q = *reinterpret_cast<const float4*>(o);
        x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
      } else {
        x[0] = o[0], x[1] = o[1], x[2] = o[2], x[3] = o[3];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(f, x[e], v[e]);
    }
    tc::st_async_v4(tc::map_to_rank(o_at + (s * out_share + idx - owner * out_share) * 4, owner),
                    __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]), tc::map_to_rank(received, owner));
  }
  for (int k = threadIdx.x; k < S * grp; k += C::kThreads) {
    const int to = k / grp, r = k - to * grp;
    const float4 v = stats[r];
    tc::st_async_v4(tc::map_to_rank(stats_at + (s * C::kHeads + r) * 16, to), __float_as_uint(v.x),
                    __float_as_uint(v.y), __float_as_uint(v.z), 0u, tc::map_to_rank(received, to));
  }
  // A CTA that gives up sends at most R + 1 limits after it began the wait that
  // ran out: that wait, and one for each place of the ring.
  bool got = false;
  for (int k = 0; k < 4 * R && !got; ++k) got = tc::mbar_wait_cluster(received, 0);
  if (!got) record_error(a.err, PA_DEVERR_TIMEOUT);
  const float4* all = reinterpret_cast<const float4*>(smem + C::kOffReceived + 16);   // [CTA][head]
  const float* parts = reinterpret_cast<const float*>(all + S * C::kHeads);           // [CTA][share]
  for (int n = threadIdx.x; n < out_n; n += C::kThreads) {
    const int r = (out_begin + n) / D, e = (out_begin + n) % D;
    float4 v[kMaxShares];
    float o[kMaxShares], M = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < kMaxShares; ++k) {
      v[k] = k < S ? all[k * C::kHeads + r] : make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
      o[k] = k < S ? parts[k * out_share + n] : 0.f;
      M = fmaxf(M, v[k].x);
    }
    float L = 0.f, LR = 0.f, acc = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxShares; ++k) {
      // (Nothing visible: all sums are 0, or NaN where the query is.)
      const float f = v[k].x == M ? 1.f : fast_exp2(v[k].x - M);
      L += f * v[k].y;
      LR += f * v[k].z;
      acc += f * o[k];
    }
    a.out[(row0 + r) * D + e] = __float2bfloat16_rn(LR == 0.f ? 0.f : acc / LR * a.out_scale);
    if (e == 0 && a.lse != nullptr)
      a.lse[row0 + r] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
  }
}

// The pool viewed 5-D, innermost first.  Rows of one column group (128 bytes,
// or 64 codes): row, tokens of a block, heads, K or V, blocks; a box is the
// 16-token K and V tiles of one head.  Rows of two: column group, tokens,
// groups, heads, 2 * block + (K or V); a box is one of the two tiles.
bool make_tile_map(CUtensorMap* map, const DecodeWindowLaunch& n) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr || 2LL * n.num_blocks > INT_MAX) return false;   // 32-bit coordinates
  const cuuint64_t el = n.fp8 ? 1 : 2, row = n.d * el, group = row < 128 ? row : 128;
  const cuuint64_t bs = n.bs, heads = n.Hkv, blocks = n.num_blocks, tok = row * heads;
  const cuuint64_t dims1[5] = {group / el, bs, heads, 2, blocks};
  const cuuint64_t strides1[4] = {tok, row, tok * bs, 2 * tok * bs};
  const cuuint64_t dims2[5] = {group / el, bs, row / group, heads, 2 * blocks};
  const cuuint64_t strides2[4] = {tok, group, row, tok * bs};
  const cuuint32_t width = static_cast<cuuint32_t>(group / el);
  const cuuint32_t box1[5] = {width, 16, 1, 2, 1}, box2[5] = {width, 16, 2, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const bool one = row == group;
  return fn(map, n.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            const_cast<void*>(n.cache), one ? dims1 : dims2, one ? strides1 : strides2,
            one ? box1 : box2, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            group == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class KV, int D, int R, int NT, int W, int MINB>
cudaError_t launch_t(const DecodeWindowLaunch& n, const WindowArgs& a, int S, cudaStream_t stream) {
  using C = WindowCfg<KV, D, R, NT, W>;
  auto kern = decode_window_kernel<KV, D, R, NT, W, MINB>;
  CUtensorMap map;
  if (!make_tile_map(&map, n)) return cudaErrorInvalidValue;
  static DeviceFlags smem_set;
  cudaError_t e = set_smem_once(
      kern, C::kSmemBytes + C::received_bytes(kMaxShares, output_share(C::kHeads * D, kMaxShares)),
      smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, n.Hkv, n.N);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes =
      C::kSmemBytes + (S > 1 ? C::received_bytes(S, a.out_share) : 0);
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
  return cudaLaunchKernelEx(&cfg, kern, map, a);
}

template <class KV, int D, int R, int NT, int MINB>
cudaError_t launch_warps(const DecodeWindowLaunch& n, const WindowArgs& a, int S, int warps,
                         cudaStream_t stream) {
  if constexpr (NT == 1)
    if (warps == 16) return launch_t<KV, D, R, NT, 16, 1>(n, a, S, stream);
  return warps == 8 ? launch_t<KV, D, R, NT, 8, 3 - NT>(n, a, S, stream)
                    : launch_t<KV, D, R, NT, 4, MINB>(n, a, S, stream);
}

}  // namespace

#ifdef PA_TEST_HOOKS
// Test builds only (not declared in pa.h).
extern "C" int pa_test_skip_decode_box(int share, int box) {
  const int2 v = make_int2(share, box);
  const int late = 0;
  return cudaMemcpyToSymbol(g_decode_skip, &v, sizeof(v)) == cudaSuccess &&
                 cudaMemcpyToSymbol(g_decode_late, &late, sizeof(late)) == cudaSuccess
             ? 0 : 3;
}
extern "C" int pa_test_late_decode_box(int share, int box) {
  const int late = 1;
  const int e = pa_test_skip_decode_box(share, box);
  return e != 0 || cudaMemcpyToSymbol(g_decode_late, &late, sizeof(late)) != cudaSuccess ? 3 : 0;
}
// What g_decode_left has counted since the last call: {issued after, on their way}.
extern "C" int pa_test_decode_left(int* two) {
  const int2 none = make_int2(0, 0);
  return cudaMemcpyFromSymbol(two, g_decode_left, sizeof(none)) == cudaSuccess &&
                 cudaMemcpyToSymbol(g_decode_left, &none, sizeof(none)) == cudaSuccess
             ? 0 : 3;
}
#endif

// CTAs per (request, kv head): as many as leave at most two per SM, up to 8,
// and at least 64 tokens to each.  More CTAs cost more than they bring, since
// each pays for its start, its merge and its cluster: 64 requests x 8 heads
// (window 1024) take 41 us on one CTA each, 49 on two, 54 on four; 8 x 8 (window
// 4096) 62 on one, 36 on two, 25 on four, 27 on eight; 1 x 8 on eight 8.1, on
// sixteen (more than a portable cluster) the same.
int decode_window_shares(int N, int Hkv, long long visible, int sm_count) {
  const long long units = static_cast<long long>(N) * Hkv;
  const long long s =
      std::min({static_cast<long long>(kMaxShares), 2LL * sm_count / units, visible / 64});
  return s < 1 ? 1 : static_cast<int>(s);
}

// Warps per CTA.  Where no SM gets a second CTA, 16 (8 for short shares, whose
// warps would have nothing to do, and for groups of 9 to 16 heads, which need the
// registers): one request x 8 heads, 512 tokens per share, 8.2 us (8.6 with 8
// warps, 13.5 with 4), 4 query heads per group 7.5 (8.3); 256 tokens 6.4 with
// either; 64 tokens 6.1 (5.0).  Else 8 where a share is long (and registers leave
// room for two such CTAs), 4 otherwise, so that twice as many CTAs are
// resident: 64 x 8 at 4100 tokens each 137.5 us with 8 (140 with 4), 128 x 8 over
// an e4m3 pool 152 (164); but 64 x 8 at 1028 tokens 43.2 (42.5), over an e4m3 pool
// 31.8 (26.8).
int decode_window_warps(long long ctas, long long share, bool wide, int sm_count) {
  if (ctas <= sm_count) return share >= 512 && !wide ? 16 : 8;
  return share >= 4096 && !wide ? 8 : 4;
}

cudaError_t launch_decode_window(const DecodeWindowLaunch& n, cudaStream_t stream) {
  WindowArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(n.q);
  a.block_table = n.block_table;
  a.seq_lens = n.seq_lens;
  a.max_blocks = n.max_blocks;
  a.Hq = n.Hq;
  a.grp = n.Hq / n.Hkv;
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
  const long long positions = static_cast<long long>(n.max_blocks) * n.bs;
  const long long visible = std::min(static_cast<long long>(n.window) + n.sinks, positions);
  a.positions = static_cast<int>(std::min(positions, INT_MAX - 64LL));
  const int S = decode_window_shares(n.N, n.Hkv, visible, n.sm_count);
  a.out_share = output_share(a.grp * n.d, S);
  const bool wide = a.grp > 8;   // groups of 9..16 heads take two n-tiles
  using dec::KvBf16;
  using dec::KvE4m3;
  const int warps = decode_window_warps(static_cast<long long>(S) * n.Hkv * n.N, visible / S,
                                        wide, n.sm_count);
  // Ring places, n-tiles and, with four warps, CTAs per SM (48 KB of ring each;
  // the two-n-tile forms are held to fewer by their registers).
  if (n.fp8) {
    if (n.d == 128)
      return wide ? launch_warps<KvE4m3<128>, 128, 3, 2, 3>(n, a, S, warps, stream)
                  : launch_warps<KvE4m3<128>, 128, 3, 1, 4>(n, a, S, warps, stream);
    return wide ? launch_warps<KvE4m3<64>, 64, 6, 2, 4>(n, a, S, warps, stream)
                : launch_warps<KvE4m3<64>, 64, 6, 1, 4>(n, a, S, warps, stream);
  }
  if (n.d == 128)
    return wide ? launch_warps<KvBf16<128>, 128, 3, 2, 2>(n, a, S, warps, stream)
                : launch_warps<KvBf16<128>, 128, 3, 1, 4>(n, a, S, warps, stream);
  return wide ? launch_warps<KvBf16<64>, 64, 3, 2, 3>(n, a, S, warps, stream)
              : launch_warps<KvBf16<64>, 64, 3, 1, 4>(n, a, S, warps, stream);
}

}  // namespace pa
