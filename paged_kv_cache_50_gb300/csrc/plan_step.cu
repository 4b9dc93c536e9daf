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
// no CTA waits for another: every CTA owns 1024 tokens and repeats the prefix
// sums over the requests up to its tokens, 1024 requests per step, from L2
// (8 bytes per request; 65535 requests are 64 steps).
// Sums saturate at INT_MAX (min(a + b, INT_MAX) is associative for
// non-negative values), so bad lengths can neither wrap nor index anything.
#include <climits>

#include "pa_common.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kPlanThreads = 1024;

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
};

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanArgs a) {
  __shared__ uint32_t s_tok[kPlanThreads + 1];   // first token of each request of the step
  __shared__ uint32_t s_blk[kPlanThreads];       // its first new block, counted from 0
  __shared__ int s_ctx[kPlanThreads];
  __shared__ uint32_t s_wt[32], s_wb[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t t0 = blockIdx.x * static_cast<uint32_t>(kPlanThreads);
  const uint32_t t = t0 + tid;   // this thread's token
  const bool mine = t < static_cast<uint32_t>(a.max_tokens);
  const int start = a.free_start != nullptr ? __ldg(a.free_start) : 0;
  uint32_t tok = 0, blk = 0;     // tokens and new blocks of the requests before the step
  bool done = false;
  int bad = 0;
  const int steps = (a.num_seqs + kPlanThreads - 1) / kPlanThreads;
  for (int step = 0; step < steps; ++step) {
    // Step k's per-request outputs are written by CTA k, the last CTA takes
    // the rest.
    const bool owner = blockIdx.x == min(static_cast<unsigned>(step), gridDim.x - 1);
    // Past this CTA's tokens and requests: nothing left to do.
    if (tok >= t0 + kPlanThreads && blockIdx.x != gridDim.x - 1 &&
        (blockIdx.x < static_cast<unsigned>(step) || blockIdx.x >= static_cast<unsigned>(steps)))
      break;
    const int i = step * kPlanThreads + tid;
    int ctx = 0, q = 0;
    uint32_t fresh = 0;
    if (i < a.num_seqs) {
      ctx = __ldg(a.context_lens + i);
      q = __ldg(a.query_lens + i);
      if (ctx < 0 || q < 0) bad |= PA_DEVERR_LENGTH;
      ctx = max(ctx, 0);
      q = max(q, 0);
      if (q > INT_MAX - ctx) {
        bad |= PA_DEVERR_LENGTH;
        q = INT_MAX - ctx;
      }
      // ceil(x / bs) = x / bs + (x % bs != 0): no overflow near INT_MAX.
      const int seq = ctx + q;
      const int have = div_bs(ctx, a.bs, a.bs_log2) + (mod_bs(ctx, a.bs, a.bs_log2) != 0);
      const int need = div_bs(seq, a.bs, a.bs_log2) + (mod_bs(seq, a.bs, a.bs_log2) != 0);
      fresh = static_cast<uint32_t>(need - have);
    }
    uint32_t xt = q, xb = fresh;   // inclusive scans over the step's requests
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
      uint32_t wt = s_wt[lane], wb = s_wb[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t yt = __shfl_up_sync(0xffffffffu, wt, o);
        const uint32_t yb = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
          wt = sat_add(wt, yt);
          wb = sat_add(wb, yb);
        }
      }
      st = __shfl_sync(0xffffffffu, wt, 31);
      sb = __shfl_sync(0xffffffffu, wb, 31);
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
    s_tok[tid] = et;
    s_blk[tid] = eb;
    s_ctx[tid] = ctx;
    if (tid == 0) s_tok[kPlanThreads] = tok_end;
    if (owner && i < a.num_seqs) {
      a.query_start_loc[i] = static_cast<int32_t>(et);
      a.seq_lens[i] = ctx + q;
    }
    __syncthreads();
    if (mine && !done && t < tok_end) {
      done = true;
      // The last request that starts at or before t (requests without new
      // tokens share their start with the next one).
      int lo = 0, hi = kPlanThreads - 1;
#pragma unroll
      for (int k = 0; k < 10; ++k) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tok[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int r = step * kPlanThreads + lo;   // < num_seqs: the padding of a step starts at tok_end > t
      const int c = s_ctx[lo];
      const int pos = c + static_cast<int>(t - s_tok[lo]);
      const int b = div_bs(pos, a.bs, a.bs_log2), off = mod_bs(pos, a.bs, a.bs_log2);
      const int have = div_bs(c, a.bs, a.bs_log2) + (mod_bs(c, a.bs, a.bs_log2) != 0);
      int32_t* entry = a.block_table + static_cast<int64_t>(r) * a.max_blocks + b;
      int id = -1;
      if (b < have) {
        // The part-filled last block of the context.
        if (b < a.max_blocks) {
          id = *entry;
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
          id = __ldg(a.free_blocks + f);
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
      a.query_start_loc[a.num_seqs] = static_cast<int32_t>(tok);
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
                   query_start_loc, seq_lens, positions, slot_mapping, totals, err};
  const unsigned grid = max_tokens > 0
                            ? static_cast<unsigned>((max_tokens - 1) / kPlanThreads + 1) : 1u;
  return launch_pdl(plan_step_kernel, dim3(grid), dim3(kPlanThreads), 0, stream, a);
}

}  // namespace pa
