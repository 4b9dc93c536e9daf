// The step plan: block tables, slot maps and positions of a serving step from
// the requests' lengths ("Attention Backends", section "What 'paged attention'
// requires of a kernel": block_table and slot_mapping; slot = block_table[pos
// / bs] * bs + pos % bs, section "Code").
//
// Mathematics: two exclusive prefix sums over the requests -- of the new
// tokens (query_start_loc) and of the new blocks ceil(seq / bs) - ceil(ctx /
// bs) (where a request's blocks start in the free list) -- and then one
// independent lookup per token.  A new block b starts at position b * bs,
// which lies among the new tokens, so the token at that position writes the
// table entry and every other token takes its block id from the free list
// itself: no token waits for a table write.
//
// Bound by latency: 131072 tokens are 1.7 MB of traffic.  So one launch, and
// no CTA waits for another: every CTA owns as many tokens as it has threads and
// repeats the prefix sums over the requests up to its tokens, from L2 (8 bytes per
// request; 65535 requests are 16 steps of 4096).  64 requests and tokens take 2.3
// us (an empty kernel 2.2), 16 requests with 18432 tokens 2.3, 4096 requests with
// 131072 tokens 4.7.
// Sums saturate at INT_MAX (min(a + b, INT_MAX) is associative for
// non-negative values), so bad lengths can neither wrap nor index anything.
#include <climits>

#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  return min(a + b, static_cast<uint32_t>(INT_MAX));   // a, b <= INT_MAX: no wrap
}

struct PlanArgs {
  const int32_t* context_lens;
  const int32_t* query_lens;
  const int32_t* free_blocks;
  const int32_t* free_start;
  int num_free, num_seqs, max_blocks, bs, bs_log2, num_blocks, max_tokens;
  int32_t* block_table;
  int32_t* query_start_loc;
  int32_t* seq_lens;
  int32_t* positions;
  int64_t* slot_mapping;
  int32_t* totals;
  int* err;
  bool vectors;   // lengths 16-byte aligned
};

// ceil(x / bs) without overflow near INT_MAX.
__device__ __forceinline__ int blocks_of(int x, const PlanArgs& a) {
  return div_bs(x, a.bs, a.bs_log2) + (mod_bs(x, a.bs, a.bs_log2) != 0);
}

// kPlanThreads: tokens of a CTA; kPer: requests of a thread in a step of the
// prefix sums.
template <int kPlanThreads, int kPer>
__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanArgs a) {
  constexpr int kStep = kPlanThreads * kPer, kWarps = kPlanThreads / 32;
  __shared__ uint32_t s_tok[kStep];   // first token of each request of the step
  __shared__ uint32_t s_blk[kStep];   // its first new block, counted from 0
  __shared__ uint32_t s_wt[kWarps], s_wb[kWarps];
  // Inputs may be the previous kernel's outputs: plain loads, no read-only path.
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t t0 = blockIdx.x * static_cast<uint32_t>(kPlanThreads);
  const uint32_t t = t0 + tid;   // this thread's token
  const bool mine = t < static_cast<uint32_t>(a.max_tokens);
  const int start = a.free_start != nullptr ? *a.free_start : 0;
  uint32_t tok = 0, blk = 0;     // tokens and new blocks of the requests before the step
  bool done = false;
  int bad = 0;
  const int steps = (a.num_seqs + kStep - 1) / kStep;
  for (int step = 0; step < steps; ++step) {
    // Step k's per-request outputs are written by CTA k, the last CTA takes the
    // rest; those of a single step of 4096, which every CTA walks, by all CTAs, a
    // warp's each (one CTA would take 0.9 us longer than the others).
    const bool owner = blockIdx.x == (kPer > 1 && steps == 1
                                          ? warp % gridDim.x
                                          : min(static_cast<unsigned>(step), gridDim.x - 1));
    // Past this CTA's tokens and requests: nothing left to do.
    if (tok >= t0 + kPlanThreads && blockIdx.x != gridDim.x - 1 &&
        (blockIdx.x < static_cast<unsigned>(step) || blockIdx.x >= static_cast<unsigned>(steps)))
      break;
    // This thread's requests, kPer in a row; xt, xb: their new tokens and
    // blocks, then the inclusive scans over the step's threads.
    const int i0 = step * kStep + tid * kPer;
    uint32_t q[kPer], fresh[kPer], xt = 0, xb = 0;
    int seq[kPer], cs[kPer], ns[kPer];
    // (A thread's four lengths by one load: 0.2 us of 4096 requests.)
    const bool whole = kPer == 4 && a.vectors && i0 + kPer <= a.num_seqs;
    if (whole) {
      const int4 c = *reinterpret_cast<const int4*>(a.context_lens + i0);
      const int4 q4 = *reinterpret_cast<const int4*>(a.query_lens + i0);
      const int cv[4] = {c.x, c.y, c.z, c.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int k = 0; k < kPer; ++k) cs[k] = cv[k % 4], ns[k] = qv[k % 4];
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        cs[k] = i0 + k < a.num_seqs ? a.context_lens[i0 + k] : 0;
        ns[k] = i0 + k < a.num_seqs ? a.query_lens[i0 + k] : 0;
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      int ctx = cs[k], n = ns[k];
      if (ctx < 0 || n < 0) bad |= PA_DEVERR_LENGTH;
      ctx = max(ctx, 0);
      n = max(n, 0);
      if (n > INT_MAX - ctx) {
        bad |= PA_DEVERR_LENGTH;
        n = INT_MAX - ctx;
      }
      seq[k] = ctx + n;
      q[k] = n;
      fresh[k] = blocks_of(seq[k], a) - blocks_of(ctx, a);
      xt = sat_add(xt, q[k]);
      xb = sat_add(xb, fresh[k]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t yt = __shfl_up_sync(0xffffffffu, xt, o);
      const uint32_t yb = __shfl_up_sync(0xffffffffu, xb, o);
      if (lane >= o) {
        xt = sat_add(xt, yt);
        xb = sat_add(xb, yb);
      }
    }
    __syncthreads();   // the last step's readers are done with shared memory
    if (lane == 31) {
      s_wt[warp] = xt;
      s_wb[warp] = xb;
    }
    __syncthreads();
    uint32_t bt = 0, bb = 0, st, sb;   // sums of the warps before, and of all warps
    {
      uint32_t wt = lane < kWarps ? s_wt[lane] : 0, wb = lane < kWarps ? s_wb[lane] : 0;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t yt = __shfl_up_sync(0xffffffffu, wt, o);
        const uint32_t yb = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
          wt = sat_add(wt, yt);
          wb = sat_add(wb, yb);
        }
      }
      st = __shfl_sync(0xffffffffu, wt, kWarps - 1);
      sb = __shfl_sync(0xffffffffu, wb, kWarps - 1);
      const uint32_t pt = __shfl_sync(0xffffffffu, wt, max(warp - 1, 0));
      const uint32_t pb = __shfl_sync(0xffffffffu, wb, max(warp - 1, 0));
      if (warp > 0) {
        bt = pt;
        bb = pb;
      }
    }
    // Exclusive sums: what stands before this request.
    uint32_t et = __shfl_up_sync(0xffffffffu, xt, 1), eb = __shfl_up_sync(0xffffffffu, xb, 1);
    if (lane == 0) et = eb = 0;
    et = sat_add(tok, sat_add(bt, et));
    eb = sat_add(blk, sat_add(bb, eb));
    const uint32_t tok_end = sat_add(tok, st);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      s_tok[tid * kPer + k] = et;
      s_blk[tid * kPer + k] = eb;
      if (owner && i0 + k < a.num_seqs) {
        // At most max_tokens: rows of a buffer of that length stay in range.
        a.query_start_loc[i0 + k] = min(static_cast<int>(et), a.max_tokens);
        a.seq_lens[i0 + k] = seq[k];
      }
      et = sat_add(et, q[k]);
      eb = sat_add(eb, fresh[k]);
    }
    __syncthreads();
    if (mine && !done && t < tok_end) {
      done = true;
      // The last request that starts at or before t (requests without new
      // tokens share their start with the next one).
      int lo = 0, hi = min(kStep, a.num_seqs - step * kStep) - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tok[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int r = step * kStep + lo;
      const int c = max(a.context_lens[r], 0);
      const int pos = c + static_cast<int>(t - s_tok[lo]);
      const int b = div_bs(pos, a.bs, a.bs_log2), off = mod_bs(pos, a.bs, a.bs_log2);
      const int have = blocks_of(c, a);
      int32_t* entry = a.block_table + static_cast<int64_t>(r) * a.max_blocks + b;
      int id = -1;
      if (b < have) {
        // The part-filled last block of the context.
        if (b < a.max_blocks) {
          // Past L1: other CTAs write entries of the same line, and a kernel that
          // is launched while this one runs must not find the line there.
          id = __ldcg(entry);
          if (id < 0 || id >= a.num_blocks) {
            bad |= PA_DEVERR_BLOCK_ID;
            id = -1;
          }
        } else {
          bad |= PA_DEVERR_LENGTH;
        }
      } else {
        const long long f = static_cast<long long>(start) + s_blk[lo] + (b - have);
        if (start < 0) {
          bad |= PA_DEVERR_LENGTH;
        } else if (f >= a.num_free) {
          bad |= PA_DEVERR_NO_BLOCKS;
        } else {
          id = a.free_blocks[f];
          if (id < 0 || id >= a.num_blocks) {
            bad |= PA_DEVERR_BLOCK_ID;
            id = -1;
          }
        }
        if (b >= a.max_blocks) {
          bad |= PA_DEVERR_LENGTH;
          id = -1;
        } else if (off == 0) {
          *entry = id;
        }
      }
      a.positions[t] = pos;
      a.slot_mapping[t] = id < 0 ? -1 : static_cast<int64_t>(id) * a.bs + off;
    }
    tok = tok_end;
    blk = sat_add(blk, sb);
  }
  if (blockIdx.x == gridDim.x - 1) {
    // The last CTA has walked every request.
    if (tid == 0) {
      a.query_start_loc[a.num_seqs] = min(static_cast<int>(tok), a.max_tokens);
      a.totals[0] = static_cast<int32_t>(tok);
      a.totals[1] = static_cast<int32_t>(sat_add(max(start, 0), blk));
      if (tok > static_cast<uint32_t>(a.max_tokens)) bad |= PA_DEVERR_LENGTH;
      if (start < 0) bad |= PA_DEVERR_LENGTH;
    }
  }
  if (mine && !done) {
    a.positions[t] = 0;
    a.slot_mapping[t] = -1;
  }
  if (bad != 0) record_error(a.err, bad);
}

}  // namespace

cudaError_t launch_plan_step(const int32_t* context_lens, const int32_t* query_lens,
                             const int32_t* free_blocks, const int32_t* free_start, int num_free,
                             int num_seqs, int max_blocks, int bs, int num_blocks, int max_tokens,
                             int32_t* block_table, int32_t* query_start_loc, int32_t* seq_lens,
                             int32_t* positions, int64_t* slot_mapping, int32_t* totals, int* err,
                             cudaStream_t stream) {
  const PlanArgs a{context_lens, query_lens, free_blocks, free_start, num_free, num_seqs,
                   max_blocks, bs, block_size_log2(bs), num_blocks, max_tokens, block_table,
                   query_start_loc, seq_lens, positions, slot_mapping, totals, err,
                   (reinterpret_cast<uintptr_t>(context_lens) |
                    reinterpret_cast<uintptr_t>(query_lens)) % 16 == 0};
  // The smallest CTA whose single step holds all requests, one to a thread (64
  // requests 2.3 us with 256 threads, 3.0 with 1024; 512 requests 2.9 with 512,
  // 3.3 with 1024); above, four requests to a thread (4096 requests 4.7 us; with
  // one to a thread in four steps 1.7 us more, with eight to one of 512 threads 4.7).
  auto launch = [&](auto kernel, int threads) {
    const unsigned grid =
        max_tokens > 0 ? static_cast<unsigned>((max_tokens - 1) / threads + 1) : 1u;
    return launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
  };
  if (num_seqs <= 256) return launch(plan_step_kernel<256, 1>, 256);
  if (num_seqs <= 512) return launch(plan_step_kernel<512, 1>, 512);
  return num_seqs <= 1024 ? launch(plan_step_kernel<1024, 1>, 1024)
                          : launch(plan_step_kernel<1024, 4>, 1024);
}

}  // namespace pa
