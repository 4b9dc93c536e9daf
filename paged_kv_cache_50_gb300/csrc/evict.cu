// Eviction from a paged cache by accumulated weights.
//
// For each request longer than the budget and each kv head, the first num_first and
// the last num_recent tokens stay, and of those between them the highest sums as far
// as the budget goes (equal ones from the lowest position on).  What stays keeps its
// order and moves to the places 0 .. budget - 1 of the request: attention over the
// cache needs nothing but the new length.  Blocks behind it go back to the free list.
//
// One cluster of up to 16 CTAs serves one (request, kv head); a CTA has a part of the
// tokens, whose ranks it keeps in shared memory.
//  1. The lowest sum that stays is found by its bits, eight at a time: a histogram
//     in each CTA's shared memory over its part, summed over the cluster.
//  2. Each warp counts what stays in its share of the part; with the offsets of the
//     warps and CTAs before it, it writes the positions to kept[], by ballots.
//  3. Rows move in steps: a CTA copies its rows of a step into a ring in shared memory
//     (cp.async), several steps ahead, and from there to their places.  A kept row's
//     source never lies before its place, and the places of a step hold sources of this
//     step and of earlier ones only: so a step is written when all CTAs have it in their
//     rings, one barrier of the cluster for each, and no other order is needed.  A thread
//     reads what it has copied itself.  Rows that stay where they are (all before the
//     first one that goes) are not touched.
// A second, small kernel writes the new lengths and pushes the blocks.
//
// Bound by HBM (each moved row is read and written once).
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "fp4.cuh"
#include "pa_launch.h"
#include "tc_common.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;   // that move rows (a CTA has more: see Ring)
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;

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

// A cached row of one head, key and value, in 16-byte vectors (kVecs) and, for the
// 4-bit pool, the key's and the value's scales (kTail bytes each): byte offsets in the
// pool of the row's first vector and (behind that) first scales, and from there of the
// others, the same for every row.
template <int ROW>   // bytes of a key (or value): 256, 128, 64
struct Plain {
  static constexpr int kVecs = 2 * ROW / 16;
  static constexpr int kTail = 0;
  static constexpr int kPer = 4, kSteps = 5;
  __device__ static __forceinline__ int64_t row(const EvictArgs& a, int64_t blk, int off, int head) {
    return ((blk * 2 * a.bs + off) * a.Hkv + head) * ROW;
  }
  __device__ static __forceinline__ int tail(int) { return 0; }
  __device__ static __forceinline__ int64_t vec(const EvictArgs& a, int v) {
    return static_cast<int64_t>(v / (ROW / 16)) * a.bs * a.Hkv * ROW + v % (ROW / 16) * 16;
  }
};
template <int D>
struct Four {
  static constexpr int kVecs = 2 * (D / 2) / 16;
  static constexpr int kTail = D / 16;
  static constexpr int kPer = 2, kSteps = 6;   // (more rows to a vector: longer lists)
  __device__ static __forceinline__ int64_t row(const EvictArgs& a, int64_t blk, int off, int head) {
    return fp4::pair_at(blk, head, off >> 4, a.Hkv, a.bs >> 4, D) + (off & 15) * (D / 2);
  }
  __device__ static __forceinline__ int tail(int off) {
    return 8 * D + (off & 15) * (D / 16 - D / 2);
  }
  __device__ static __forceinline__ int64_t vec(const EvictArgs&, int v) {
    return v / (D / 32) * fp4::tile_bytes(D) + v % (D / 32) * 16;
  }
  static constexpr int kTile = fp4::tile_bytes(D);   // from the key's to the value's
};
// What is moved: from and to (offsets in the pool, -1: not there), the position, and
// where the scales are.
struct Move {
  int64_t from, to;
  int p;
  int16_t from_tail, to_tail;
};
template <class Row>
struct Ring {
  // 16-byte vectors of a thread in a step, and steps in the ring.
  static constexpr int kPer = Row::kPer, kSteps = Row::kSteps;
  static constexpr int kRows = kThreads * kPer / Row::kVecs;   // of a CTA in a step
  static constexpr int kOffTail = kThreads * kPer * 16;
  static constexpr int kOffSum = kOffTail + kRows * 2 * Row::kTail;
  static constexpr int kStepBytes = (kOffSum + kRows * 4 + 15) / 16 * 16;
  static constexpr int kOffMoves = kSteps * kStepBytes;        // lists of kSteps + 1 steps
  static constexpr int kBytes = kOffMoves + (kSteps + 1) * kRows * static_cast<int>(sizeof(Move));
  static constexpr int kKeys = kBytes / 4;                     // ranks that fit it
  // Warps beside the kThreads that move rows: they make the lists.
  static constexpr int kAll = kThreads + (kRows + 31) / 32 * 32;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <class Row>
__global__ void __launch_bounds__(Ring<Row>::kAll, 2) evict_kernel(const __grid_constant__ EvictArgs a) {
  using R = Ring<Row>;
  constexpr int kPer = R::kPer, kSteps = R::kSteps;
  extern __shared__ __align__(16) uint8_t smem[];   // the part's ranks, then the ring
  __shared__ int hist[256];
  __shared__ int merged[256];
  __shared__ int counts[3];   // this part's tokens above the threshold, at it; first place that moves
  __shared__ int warp_counts[2][kWarps];
  __shared__ uint32_t pick[2];   // threshold's bits so far, how many at or above it are wanted
  const int kvh = blockIdx.y, i = blockIdx.z;
  const int C = gridDim.x, c = blockIdx.x;   // cluster = grid.x
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool mover = threadIdx.x < kThreads;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int seq = max(0, a.seq_lens[i]);
  const int64_t unit = static_cast<int64_t>(i) * a.Hkv + kvh;
  const float* scores = a.scores + unit * a.score_tokens;
  float* fresh = a.new_scores + unit * a.score_tokens;
  int32_t* kept = a.kept + unit * a.budget;
  const int32_t* table = a.block_table + static_cast<int64_t>(i) * a.max_blocks;
  const int tid = c * R::kAll + threadIdx.x, all = C * R::kAll;

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
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  const bool held = per <= R::kKeys;   // (else they are read again)
  if (held) {
#pragma unroll 4
    for (int p = b + threadIdx.x; p < e; p += R::kAll) keys[p - b] = rank_of(scores[p]);
  }
  auto rank_at = [&](int p) { return held ? keys[p - b] : rank_of(scores[p]); };
  uint32_t prefix = 0;
  int left = want;   // of those that share the prefix
  if (want > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (mover) hist[threadIdx.x] = 0;
      __syncthreads();
#pragma unroll 4
      for (int p = max(b, lo) + threadIdx.x; p < min(e, hi); p += R::kAll) {
        const uint32_t u = rank_at(p);
        if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      cluster.sync();
      if (mover) {
        int n = 0;
#pragma unroll 8
        for (int k = 0; k < C; ++k) n += cluster.map_shared_rank(hist, k)[threadIdx.x];
        merged[threadIdx.x] = n;
      }
      cluster.sync();   // (the parts are read before they are cleared)
      // The highest digit at which the counts from above reach `left`.
      if (warp == 0) {
        int mine = 0;   // digits 255 - 8 lane ... 248 - 8 lane
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += merged[255 - 8 * lane - k];
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (x >= left && x - mine < left) {
          int above = x - mine;
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const int digit = 255 - 8 * lane - k, n = merged[digit];
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
  } else {
    __syncthreads();   // (the ranks are there)
  }
  // What stays: first, recent, ranks above the threshold, and the first `left` at it.
  auto level = [&](int p) {   // 2: stays, 1: at the threshold, 0: goes
    if (p < lo || p >= hi) return 2;
    if (want == 0) return 0;
    const uint32_t u = rank_at(p);
    return u > prefix ? 2 : u == prefix ? 1 : 0;
  };
  // A warp's share of the part, in whole 32s.
  const int share = ((e - b + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int wb = mover ? min(e, b + warp * share) : e, we = min(e, wb + share);
  int sure = 0, at = 0;
#pragma unroll 4
  for (int p = wb + lane; p < we; p += 32) {
    const int l = level(p);
    sure += l == 2;
    at += l == 1;
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  at = __reduce_add_sync(0xffffffffu, at);
  if (mover && lane == 0) warp_counts[0][warp] = sure, warp_counts[1][warp] = at;
  __syncthreads();
  if (threadIdx.x < 2) {
    int n = 0;
    for (int w = 0; w < kWarps; ++w) n += warp_counts[threadIdx.x][w];
    counts[threadIdx.x] = n;
  } else if (threadIdx.x == 2) {
    counts[2] = INT_MAX;
  }
  cluster.sync();
  int before = 0, tied = 0;   // sure and tied tokens before this warp's
#pragma unroll 8
  for (int k = 0; k < c; ++k) {
    const int* other = cluster.map_shared_rank(counts, k);
    before += other[0];
    tied += other[1];
  }
  for (int w = 0; w < min(warp, kWarps); ++w) before += warp_counts[0][w], tied += warp_counts[1][w];
  int moved = INT_MAX;   // the first place whose row moves
#pragma unroll 2
  for (int p0 = wb; p0 < we; p0 += 32) {
    const int p = p0 + lane;
    const int l = p < we ? level(p) : 0;
    const unsigned below = (1u << lane) - 1u;
    const unsigned twos = __ballot_sync(0xffffffffu, l == 2), ones = __ballot_sync(0xffffffffu, l == 1);
    const int t = tied + __popc(ones & below);
    const int j = before + __popc(twos & below) + min(t, left);
    if (l == 2 || (l == 1 && t < left)) {
      kept[j] = p;
      if (j != p) moved = min(moved, j);
    }
    before += __popc(twos);
    tied += __popc(ones);
  }
  moved = __reduce_min_sync(0xffffffffu, moved);
  if (lane == 0 && moved != INT_MAX) atomicMin(&counts[2], moved);
  cluster.sync();   // kept[] is complete, and seen by the cluster; the ranks are not needed

  // ------------------------------------------------------------ rows
  int from = INT_MAX;
#pragma unroll 8
  for (int k = 0; k < C; ++k) from = min(from, cluster.map_shared_rank(counts, k)[2]);
  from = min(from, a.budget);
  // Step s, row q of this CTA: place from + (s C + c) kRows + q.  The warps behind the
  // movers make the lists, a thread for each row: a step's position, then its blocks,
  // then its addresses, each a turn of the loop after the one before, so that none is
  // waited for.
  const uint32_t ring = smem_u32(smem);
  Move* moves = reinterpret_cast<Move*>(smem + R::kOffMoves);
  const int r = threadIdx.x / Row::kVecs, v = threadIdx.x % Row::kVecs;
  constexpr int kPass = kThreads / Row::kVecs;   // rows that the threads cover at once
  const int steps = (a.budget - from + C * R::kRows - 1) / (C * R::kRows);
  const int q0 = static_cast<int>(threadIdx.x) - kThreads;
  auto place = [&](int s) { return from + (s * C + c) * R::kRows + q0; };
  int p1 = -1;                      // of the step after the next to be listed
  int p2 = -1, sb = -1, db = -1;    // of the next
  auto list = [&](int s) {          // the list of step s, blocks of s + 1, positions of s + 2
    if (s >= 0) {
      Move m{-1, -1, p2, 0, 0};
      if (p2 >= 0) {
        const int j = place(s);
        if (sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks) {
          const int so = mod_bs(p2, a.bs, a.bs_log2), dof = mod_bs(j, a.bs, a.bs_log2);
          m.from = Row::row(a, sb, so, kvh);
          m.to = Row::row(a, db, dof, kvh);
          m.from_tail = static_cast<int16_t>(Row::tail(so));
          m.to_tail = static_cast<int16_t>(Row::tail(dof));
        } else {
          record_error(a.err, PA_DEVERR_BLOCK_ID);
        }
      }
      moves[s % (kSteps + 1) * R::kRows + q0] = m;
    }
    p2 = p1;
    if (p2 >= 0) {
      sb = table[div_bs(p2, a.bs, a.bs_log2)];
      db = table[div_bs(place(s + 1), a.bs, a.bs_log2)];
    }
    const int j = place(s + 2);
    p1 = s + 2 < steps && j < a.budget ? kept[j] : -1;
  };
  const int64_t mine = Row::vec(a, v);
  auto fetch = [&](int s) {
    const uint32_t to = ring + s % kSteps * R::kStepBytes;
    const Move* m = moves + s % (kSteps + 1) * R::kRows;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = k * kPass + r;
      const int64_t src = m[q].from;
      if (v == 0 && m[q].p >= 0) copy_async<4>(to + R::kOffSum + q * 4, scores + m[q].p);
      if (src < 0) continue;
      cp_async_16(to + (k * kThreads + threadIdx.x) * 16, a.cache + src + mine, 16);
      if constexpr (Row::kTail > 0)
        if (v < 2)
          copy_async<Row::kTail>(to + R::kOffTail + (q * 2 + v) * Row::kTail,
                                 a.cache + src + m[q].from_tail + v * Row::kTile);
    }
  };
  if (!mover) {
#pragma unroll 1
    for (int s = -2; s < kSteps; ++s) list(s);
  }
  __syncthreads();
  if (mover) {
#pragma unroll 1
    for (int s = 0; s < kSteps - 1; ++s) {
      if (s < steps) fetch(s);
      cp_async_commit();
    }
  }
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    cp_async_wait<kSteps - 2>();
    // Every row of the step has been read.  (Nothing is published: what has been read
    // is in shared memory, and may be written over.)
    if (C > 1) {
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      tc::cluster_wait();
    }
    __syncthreads();   // (and the next list is there)
    if (!mover) {
      list(s + kSteps);
      continue;
    }
    const uint8_t* held_step = smem + s % kSteps * R::kStepBytes;
    const Move* m = moves + s % (kSteps + 1) * R::kRows;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = k * kPass + r;
      const int64_t dst = m[q].to;
      if (v == 0 && m[q].p >= 0)
        fresh[from + (s * C + c) * R::kRows + q] =
            *reinterpret_cast<const float*>(held_step + R::kOffSum + q * 4);
      if (dst < 0) continue;
      *reinterpret_cast<uint4*>(a.cache + dst + mine) =
          *reinterpret_cast<const uint4*>(held_step + (k * kThreads + threadIdx.x) * 16);
      if constexpr (Row::kTail > 0)
        if (v < 2) {
          uint8_t* to = a.cache + dst + m[q].to_tail + v * Row::kTile;
          const uint8_t* got = held_step + R::kOffTail + (q * 2 + v) * Row::kTail;
          if constexpr (Row::kTail == 8)
            *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(got);
          else
            *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(got);
        }
    }
    if (s + kSteps - 1 < steps) fetch(s + kSteps - 1);
    cp_async_commit();
  }
  if (fresh != scores)
    for (int j = tid; j < from; j += all) fresh[j] = scores[j];
  // (The sums behind the budget have been read: by the last step's barrier, or, where no
  // row moved, there was none to read.)
  const int64_t clear = fresh != scores ? a.score_tokens : static_cast<int64_t>(seq);
  for (int64_t p = a.budget + tid; p < clear; p += all) fresh[p] = 0.f;
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
// One cluster, whose CTAs each sum all requests' blocks and then take a range of them:
// lengths may be updated in place, so nothing is written before all have read them.
constexpr int kBlockCtas = 8;
constexpr int kBlockThreads = 1024;
__global__ void __launch_bounds__(kBlockThreads) evict_blocks_kernel(
    const __grid_constant__ BlocksArgs a) {
  __shared__ int sums[32];
  __shared__ unsigned long long totals[2];   // all blocks; those of requests before the range
  __shared__ int list[3][kBlockThreads];     // of a round's requests: blocks, first column, place
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 2) totals[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto ceil_bs = [&](int x) { return x > 0 ? div_bs(x - 1, a.bs, a.bs_log2) + 1 : 0; };
  auto lens = [&](int i, int& seq, int& keep) {
    seq = max(0, a.seq_lens[i]);
    const bool refused = seq > a.score_tokens || seq > static_cast<int64_t>(a.max_blocks) * a.bs;
    keep = refused ? seq : min(seq, a.budget);
    return refused ? 0 : ceil_bs(seq) - ceil_bs(keep);
  };
  const int per = (a.num_seqs + kBlockCtas - 1) / kBlockCtas;
  const int r0 = min(a.num_seqs, static_cast<int>(blockIdx.x) * per), r1 = min(a.num_seqs, r0 + per);
  unsigned long long mine = 0, early = 0;
  for (int i = threadIdx.x; i < a.num_seqs; i += kBlockThreads) {
    int seq, keep;
    const int n = lens(i, seq, keep);
    mine += n;
    if (i < r0) early += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine += __shfl_xor_sync(0xffffffffu, mine, o);
    early += __shfl_xor_sync(0xffffffffu, early, o);
  }
  if (lane == 0 && mine != 0) atomicAdd(&totals[0], mine);
  if (lane == 0 && early != 0) atomicAdd(&totals[1], early);
  const int start = a.free_start != nullptr ? *a.free_start : 0;
  __syncthreads();
  const long long total = static_cast<long long>(totals[0]);
  const bool room = a.free_blocks != nullptr && start >= total && start <= a.num_free;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.free_blocks != nullptr && total > 0 && !room)
    record_error(a.err, PA_DEVERR_LENGTH);
  int before = room ? static_cast<int>(start - total + static_cast<long long>(totals[1])) : 0;
  cluster.sync();
  for (int i0 = r0; i0 < r1; i0 += kBlockThreads) {
    const int i = i0 + threadIdx.x, count = min(kBlockThreads, r1 - i0);
    int seq = 0, keep = 0, n = 0;
    if (i < r1) n = lens(i, seq, keep);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int base = before;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) base += sums[w];
      before += sums[w];
    }
    list[0][threadIdx.x] = n;
    list[1][threadIdx.x] = ceil_bs(keep);
    list[2][threadIdx.x] = base + x - n;
    if (i < r1) a.new_lens[i] = keep;
    __syncthreads();
    // A request's blocks are copied by a warp, or, where the requests are few, by all.
    const bool few = count < 32;
    const int width = few ? kBlockThreads : 32;
    if (room)
      for (int k = few ? 0 : warp; k < count; k += few ? 1 : 32) {
        const int cols = list[0][k], to = list[2][k];
        const int32_t* row = a.block_table + static_cast<int64_t>(i0 + k) * a.max_blocks + list[1][k];
#pragma unroll 4
        for (int q = few ? threadIdx.x : lane; q < cols; q += width) {
          const int blk = row[q];
          if (blk < 0 || blk >= a.num_blocks) record_error(a.err, PA_DEVERR_BLOCK_ID);
          a.free_blocks[to + q] = blk;
        }
      }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.new_free_start != nullptr)
    *a.new_free_start = room ? static_cast<int>(start - total) : start;
}

// Whether clusters of 16 are there to be had (they are not portable).
template <class Row>
bool wide_clusters() {
  static std::mutex mu;
  static int known[64] = {};   // 1: yes, 2: no
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    known[dev] = 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCtas);
    cfg.blockDim = dim3(Ring<Row>::kAll);
    cfg.dynamicSmemBytes = Ring<Row>::kBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(evict_kernel<Row>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
            cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, evict_kernel<Row>, &cfg) == cudaSuccess) {
      if (n >= 4) known[dev] = 1;
    } else {
      cudaGetLastError();   // (a refused size is no error of the call)
    }
  }
  return known[dev] == 1;
}

template <class Row>
cudaError_t launch_rows(const EvictArgs& a, int N, int sm_count, cudaStream_t stream) {
  static DeviceFlags smem_set;
  cudaError_t e = set_smem_once(evict_kernel<Row>, Ring<Row>::kBytes, smem_set);
  if (e != cudaSuccess) return e;
  // CTAs per (request, kv head): a power of two, as many as leave eight CTAs for each SM
  // (four rounds of two), but none with less than a step of rows.
  const long long units = static_cast<long long>(N) * a.Hkv;
  const int most = wide_clusters<Row>() ? kMaxCtas : 8;
  int C = 1;
  while (C < most && 2 * C * units <= 8LL * sm_count && 2LL * C * Ring<Row>::kRows <= a.budget) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, a.Hkv, N);
  cfg.blockDim = dim3(Ring<Row>::kAll);
  cfg.dynamicSmemBytes = Ring<Row>::kBytes;
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
  cudaError_t e;
  if (n.four)
    e = n.d == 128 ? launch_rows<Four<128>>(a, n.N, n.sm_count, stream)
                   : launch_rows<Four<64>>(a, n.N, n.sm_count, stream);
  else if (n.row_bytes == 256)
    e = launch_rows<Plain<256>>(a, n.N, n.sm_count, stream);
  else if (n.row_bytes == 128)
    e = launch_rows<Plain<128>>(a, n.N, n.sm_count, stream);
  else
    e = launch_rows<Plain<64>>(a, n.N, n.sm_count, stream);
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBlockCtas);
  cfg.blockDim = dim3(kBlockThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kBlockCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_blocks_kernel, f);
}

}  // namespace pa
