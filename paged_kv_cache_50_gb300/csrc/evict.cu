// Eviction from a paged cache by accumulated weights.
//
// For each request longer than the budget and each kv head, the first num_first and
// the last num_recent tokens stay, and of those between them the highest sums as far
// as the budget goes (equal ones from the lowest position on).  What stays keeps its
// order and moves to the places 0 .. budget - 1 of the request: attention over the
// cache needs nothing but the new length.  Blocks behind it go back to the free list.
//
// One cluster of up to 8 CTAs serves one (request, kv head).
//  1. The lowest sum that stays is found by its bits, eight at a time: a histogram
//     in each CTA's shared memory over its part of the tokens, summed over the cluster.
//  2. Each CTA counts what stays in its part; the parts' offsets come from the
//     cluster, and the positions are written to kept[].
//  3. Rows move in steps of kRows per CTA.  A kept row's source never lies before its
//     place, and places of a step only hold sources of this step and of earlier ones:
//     so a step's rows are all read (into registers) before any is written, with one
//     barrier of the cluster between, and no other order is needed.  Rows that stay
//     where they are (all before the first one that goes) are not touched.
// A second, small kernel writes the new lengths and pushes the blocks.
//
// Bound by HBM (each moved row is read and written once) for batches; the selection
// reads the sums four times from L2.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct EvictArgs {
  uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* scores;
  float* new_scores;
  int32_t* kept;
  int* err;
  int max_blocks, Hkv, bs, bs_log2, num_blocks;
  int64_t score_tokens;
  int budget, recent, first;
  int d;
};

// Sums in an order of unsigned integers; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A cached row of one head in 16-byte vectors (kVecs) and, for the 4-bit pool, the
// two rows' scales (kTail words).
template <int ROW>   // bytes of a key (or value): 256, 128, 64; 4-bit: codes 64, 32
struct Plain {
  static constexpr int kVecs = 2 * ROW / 16;   // keys and values
  static constexpr int kTail = 0;
  __device__ static __forceinline__ uint8_t* vec(const EvictArgs& a, int64_t blk, int off, int head,
                                                 int v) {
    const int kv = v / (ROW / 16), c = v % (ROW / 16);
    return a.cache + (((blk * 2 + kv) * a.bs + off) * a.Hkv + head) * ROW + c * 16;
  }
  __device__ static __forceinline__ uint8_t* tail(const EvictArgs& a, int64_t, int, int, int) {
    return a.cache;
  }
};
template <int D>
struct Four {
  static constexpr int kVecs = 2 * (D / 2) / 16;
  static constexpr int kTail = 2 * (D / 16) / 4;   // words
  __device__ static __forceinline__ uint8_t* vec(const EvictArgs& a, int64_t blk, int off, int head,
                                                 int v) {
    const int kv = v / (D / 32), c = v % (D / 32);
    return a.cache + fp4::pair_at(blk, head, off >> 4, a.Hkv, a.bs >> 4, D) +
           kv * fp4::tile_bytes(D) + (off & 15) * (D / 2) + c * 16;
  }
  __device__ static __forceinline__ uint8_t* tail(const EvictArgs& a, int64_t blk, int off, int head,
                                                  int w) {
    const int kv = w / (D / 64), c = w % (D / 64);
    return a.cache + fp4::pair_at(blk, head, off >> 4, a.Hkv, a.bs >> 4, D) +
           kv * fp4::tile_bytes(D) + 8 * D + (off & 15) * (D / 16) + c * 4;
  }
};

// Exclusive prefix sum of v over the CTA, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int y = warp_sums[w];
    if (w < warp) before += y;
    total += y;
  }
  __syncthreads();
  return before + x - v;
}

template <class Row>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int merged[256];
  __shared__ int warp_sums[kWarps];
  __shared__ int counts[3];   // this part's tokens above the threshold, at it; first place that moves
  __shared__ uint32_t pick[2];   // threshold's bits so far, how many at or above it are wanted
  const int kvh = blockIdx.y, i = blockIdx.z;
  const int C = gridDim.x, c = blockIdx.x;   // cluster = grid.x
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int seq = max(0, a.seq_lens[i]);
  const int64_t unit = static_cast<int64_t>(i) * a.Hkv + kvh;
  const float* scores = a.scores + unit * a.score_tokens;
  float* fresh = a.new_scores + unit * a.score_tokens;
  int32_t* kept = a.kept + unit * a.budget;
  const int32_t* table = a.block_table + static_cast<int64_t>(i) * a.max_blocks;
  const int tid = c * kThreads + threadIdx.x, all = C * kThreads;

  // A length past the sums or the table: nothing is done to the request.
  const bool refused = seq > a.score_tokens || seq > static_cast<int64_t>(a.max_blocks) * a.bs;
  if (refused && tid == 0 && kvh == 0) record_error(a.err, PA_DEVERR_LENGTH);
  if (seq <= a.budget || refused) {
    // All stays (the same decision in all CTAs of the cluster).
    const int n = min(seq, a.budget);
    for (int p = tid; p < a.budget; p += all) kept[p] = p < n ? p : -1;
    if (fresh != scores)
      for (int64_t p = tid; p < a.score_tokens; p += all) fresh[p] = p < seq ? scores[p] : 0.f;
    return;
  }

  // ------------------------------------------------------------ selection
  // Candidates [lo, hi), of which `want` stay; this CTA's part [b, e) of all positions.
  const int lo = a.first, hi = seq - a.recent, want = a.budget - a.first - a.recent;
  const int per = (seq + C - 1) / C;
  const int b = min(seq, c * per), e = min(seq, b + per);
  uint32_t prefix = 0;
  int left = want;   // of those that share the prefix
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int k = threadIdx.x; k < 256; k += kThreads) hist[k] = 0;
      __syncthreads();
      for (int p = max(b, lo) + threadIdx.x; p < min(e, hi); p += kThreads) {
        const uint32_t u = rank_of(scores[p]);
        if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      cluster.sync();
      if (threadIdx.x < 256) {
        int n = 0;
        for (int k = 0; k < C; ++k) n += cluster.map_shared_rank(hist, k)[threadIdx.x];
        merged[threadIdx.x] = n;
      }
      cluster.sync();   // (the parts are read before they are cleared)
      // The highest digit at which the counts from above reach `left`.
      if (threadIdx.x < 32) {
        int mine = 0;   // digits 255 - 8 lane ... 248 - 8 lane
        for (int k = 0; k < 8; ++k) mine += merged[255 - 8 * threadIdx.x - k];
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (static_cast<int>(threadIdx.x) >= o) x += y;
        }
        if (x >= left && x - mine < left) {
          int above = x - mine;
          for (int k = 0; k < 8; ++k) {
            const int digit = 255 - 8 * threadIdx.x - k, n = merged[digit];
            if (above + n >= left) {
              pick[0] = prefix | (static_cast<uint32_t>(digit) << shift);
              pick[1] = left - above;
              break;
            }
            above += n;
          }
        }
      }
      __syncthreads();
      prefix = pick[0];
      left = static_cast<int>(pick[1]);
    }
  }
  // What stays: first, recent, ranks above the threshold, and the first `left` at it.
  if (threadIdx.x < 3) counts[threadIdx.x] = threadIdx.x == 2 ? INT_MAX : 0;
  __syncthreads();
  auto level = [&](int p) {   // 2: stays, 1: at the threshold, 0: goes
    if (p < lo || p >= hi) return 2;
    if (want == 0) return 0;
    const uint32_t u = rank_of(scores[p]);
    return u > prefix ? 2 : u == prefix ? 1 : 0;
  };
  int sure = 0, at = 0;
  for (int p = b + threadIdx.x; p < e; p += kThreads) {
    const int l = level(p);
    sure += l == 2;
    at += l == 1;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sure += __shfl_xor_sync(0xffffffffu, sure, o);
    at += __shfl_xor_sync(0xffffffffu, at, o);
  }
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&counts[0], sure);
    atomicAdd(&counts[1], at);
  }
  cluster.sync();
  int place = 0, tied = 0;   // before this part
  for (int k = 0; k < c; ++k) {
    const int* other = cluster.map_shared_rank(counts, k);
    place += other[0];
    tied += other[1];
  }
  place += min(tied, left);
  for (int p0 = b; p0 < e; p0 += kThreads) {
    const int p = p0 + threadIdx.x;
    const int l = p < e ? level(p) : 0;
    int n1, n2;
    const int t = block_scan(l == 1, warp_sums, n1);
    const bool stays = l == 2 || (l == 1 && tied + t < left);
    const int j = block_scan(stays, warp_sums, n2);
    if (stays) {
      kept[place + j] = p;
      if (place + j != p) atomicMin(&counts[2], place + j);
    }
    place += n2;
    tied += n1;
  }
  cluster.sync();   // kept[] is complete, and seen by the cluster

  // ------------------------------------------------------------ rows
  int from = INT_MAX;   // the first place whose row moves
  for (int k = 0; k < C; ++k) from = min(from, cluster.map_shared_rank(counts, k)[2]);
  // Sums, in the same steps as rows below where they may share memory.
  constexpr int kLanes = Row::kVecs;                  // threads of a row
  constexpr int kRows = kThreads / kLanes;            // rows of a round
  constexpr int kRounds = 8;                          // rounds of a step
  const int r = threadIdx.x / kLanes, v = threadIdx.x % kLanes;
  const int step = C * kRows * kRounds;
  for (int j0 = min(from, a.budget); j0 < a.budget; j0 += step) {
    uint4 row[kRounds];
    uint32_t tail[kRounds];
    float sum[kRounds];
    uint8_t* to[kRounds];
    uint8_t* to_tail[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int j = j0 + (k * C + c) * kRows + r;
      to[k] = nullptr;
      if (j < a.budget) {
        const int p = kept[j];
        sum[k] = scores[p];
        const int sb = table[div_bs(p, a.bs, a.bs_log2)], db = table[div_bs(j, a.bs, a.bs_log2)];
        const int so = mod_bs(p, a.bs, a.bs_log2), dof = mod_bs(j, a.bs, a.bs_log2);
        if (sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks) {
          row[k] = *reinterpret_cast<const uint4*>(Row::vec(a, sb, so, kvh, v));
          to[k] = Row::vec(a, db, dof, kvh, v);
          if constexpr (Row::kTail > 0) {
            if (v < Row::kTail) {
              tail[k] = *reinterpret_cast<const uint32_t*>(Row::tail(a, sb, so, kvh, v));
              to_tail[k] = Row::tail(a, db, dof, kvh, v);
            }
          }
        } else if (v == 0) {
          record_error(a.err, PA_DEVERR_BLOCK_ID);
        }
      }
    }
    cluster.sync();   // every row of the step has been read
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int j = j0 + (k * C + c) * kRows + r;
      if (j < a.budget && v == 0) fresh[j] = sum[k];
      if (to[k] != nullptr) {
        *reinterpret_cast<uint4*>(to[k]) = row[k];
        if constexpr (Row::kTail > 0)
          if (v < Row::kTail) *reinterpret_cast<uint32_t*>(to_tail[k]) = tail[k];
      }
    }
  }
  if (fresh != scores)
    for (int j = tid; j < min(from, a.budget); j += all) fresh[j] = scores[j];
  // (The sums behind the budget have been read: by the last step's barrier, or, where no
  // row moved, there was none to read.)
  for (int64_t p = a.budget + tid; p < (fresh != scores ? a.score_tokens : static_cast<int64_t>(seq));
       p += all)
    fresh[p] = 0.f;
  cluster.sync();   // no CTA leaves while others read its shared memory
}

struct BlocksArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* free_blocks;      // null: blocks are not given back
  const int32_t* free_start;
  int32_t* new_free_start;
  int* err;
  int num_seqs, max_blocks, bs, bs_log2, num_free, num_blocks, budget;
  int64_t score_tokens;
};

// New lengths; the blocks behind them go in front of free_start, by request and column.
// One CTA: a scan over the requests, 1024 at a time.
__global__ void __launch_bounds__(1024) evict_blocks_kernel(const __grid_constant__ BlocksArgs a) {
  __shared__ int sums[32];
  __shared__ unsigned long long total_s;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto ceil_bs = [&](int x) { return x > 0 ? div_bs(x - 1, a.bs, a.bs_log2) + 1 : 0; };
  auto lens = [&](int i, int& seq, int& keep) {
    seq = i < a.num_seqs ? max(0, a.seq_lens[i]) : 0;
    const bool refused = seq > a.score_tokens || seq > static_cast<int64_t>(a.max_blocks) * a.bs;
    keep = refused ? seq : min(seq, a.budget);
    return refused ? 0 : ceil_bs(seq) - ceil_bs(keep);
  };
  if (threadIdx.x == 0) total_s = 0;
  __syncthreads();
  unsigned long long mine = 0;
  for (int i = threadIdx.x; i < a.num_seqs; i += 1024) {
    int seq, keep;
    mine += lens(i, seq, keep);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0 && mine != 0) atomicAdd(&total_s, mine);
  __syncthreads();
  const long long total = static_cast<long long>(total_s);
  const int start = a.free_start != nullptr ? *a.free_start : 0;
  const bool room = a.free_blocks != nullptr && start >= total && start <= a.num_free;
  if (threadIdx.x == 0 && a.free_blocks != nullptr && total > 0 && !room)
    record_error(a.err, PA_DEVERR_LENGTH);
  int before = room ? static_cast<int>(start - total) : 0;
  __syncthreads();
  for (int i0 = 0; i0 < a.num_seqs; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    int seq, keep;
    const int n = lens(i, seq, keep);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int base = before, chunk = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) base += sums[w];
      chunk += sums[w];
    }
    __syncthreads();
    // A warp's requests in turn, their columns by its lanes.
    const int at = base + x - n, col0 = ceil_bs(keep);
    if (room)
      for (int k = 0; k < 32; ++k) {
        const int cols = __shfl_sync(0xffffffffu, n, k);
        const int to = __shfl_sync(0xffffffffu, at, k), from = __shfl_sync(0xffffffffu, col0, k);
        const int64_t row = static_cast<int64_t>(i0 + warp * 32 + k) * a.max_blocks + from;
        for (int q = lane; q < cols; q += 32) {
          const int blk = a.block_table[row + q];
          if (blk < 0 || blk >= a.num_blocks) record_error(a.err, PA_DEVERR_BLOCK_ID);
          a.free_blocks[to + q] = blk;
        }
      }
    if (i < a.num_seqs) a.new_lens[i] = keep;
    before += chunk;
  }
  if (threadIdx.x == 0 && a.new_free_start != nullptr) *a.new_free_start = room ? static_cast<int>(start - total) : start;
}

template <class Row>
cudaError_t launch_rows(const EvictArgs& a, int N, int C, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, a.Hkv, N);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<Row>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& n, cudaStream_t stream) {
  EvictArgs a{};
  a.cache = static_cast<uint8_t*>(n.cache);
  a.block_table = n.block_table;
  a.seq_lens = n.seq_lens;
  a.scores = n.scores;
  a.new_scores = n.new_scores;
  a.kept = n.kept;
  a.err = n.err;
  a.max_blocks = n.max_blocks;
  a.Hkv = n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  a.num_blocks = n.num_blocks;
  a.score_tokens = n.score_tokens;
  a.budget = n.budget;
  a.recent = n.recent;
  a.first = n.first;
  a.d = n.d;
  // CTAs per (request, kv head): as many as leave two per SM, a power of two up to 8.
  const long long units = static_cast<long long>(n.N) * n.Hkv;
  int C = 1;
  while (C < 8 && 2 * C * units <= 2LL * n.sm_count) C *= 2;
  cudaError_t e;
  if (n.four)
    e = n.d == 128 ? launch_rows<Four<128>>(a, n.N, C, stream)
                   : launch_rows<Four<64>>(a, n.N, C, stream);
  else if (n.row_bytes == 256)
    e = launch_rows<Plain<256>>(a, n.N, C, stream);
  else if (n.row_bytes == 128)
    e = launch_rows<Plain<128>>(a, n.N, C, stream);
  else
    e = launch_rows<Plain<64>>(a, n.N, C, stream);
  if (e != cudaSuccess) return e;
  BlocksArgs f{};
  f.block_table = n.block_table;
  f.seq_lens = n.seq_lens;
  f.new_lens = n.new_lens;
  f.free_blocks = n.free_blocks;
  f.free_start = n.free_start;
  f.new_free_start = n.new_free_start;
  f.err = n.err;
  f.num_seqs = n.N;
  f.max_blocks = n.max_blocks;
  f.bs = n.bs;
  f.bs_log2 = a.bs_log2;
  f.num_free = n.num_free;
  f.num_blocks = n.num_blocks;
  f.budget = n.budget;
  f.score_tokens = n.score_tokens;
  return launch_pdl(evict_blocks_kernel, dim3(1), dim3(1024), 0, stream, f);
}

}  // namespace pa
