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
//     in each CTA's shared memory over its part, summed over the cluster, one barrier of
//     the cluster for each (two histograms in turn).
//  2. Each warp counts what stays in its share of the part; with the offsets of the
//     warps and CTAs before it, it writes the positions to kept[], by ballots.
//  3. Rows move in steps: a CTA copies its rows of a step into a ring in shared memory
//     (cp.async), several steps ahead, and from there to their places, by lists of
//     addresses that warps of their own make.  A kept row's source never lies before its
//     place, and the places of a step hold sources of this step and of earlier ones only:
//     so a step is written when all CTAs have it in their rings, one barrier of the
//     cluster for each, and no other order is needed.  A thread reads what it has copied
//     itself.  Rows that stay where they are (all before the first one that goes) are not
//     touched.
// A second, small kernel writes the new lengths and pushes the blocks, beside the first
// where SMs are free.
//
// Bound by HBM in the long run (each moved row is read and written once): 64 requests in
// bf16 move 667 MB in 154 us.  One long stream has no more than 96 CTAs (8 clusters of 12)
// and is bound by their chains of barriers: 52 us, of them 4 for the ranks' loads, 11 for
// the four histograms, 8 for the list and the first rows, 21 for the rows.
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

constexpr int kMaxCtas = 16;
constexpr int kMaxWarps = 24;

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
// others, the same for every row.  kMovers threads move kPer vectors each in a step, with
// kSteps steps in flight, kCtas CTAs to an SM: a step's time is the chain of a warp's
// instructions, so threads are many and steps are large.  (64 requests in bf16: 2 CTAs
// with 5 steps 185 us, 3 with 4: 160, 4 with 3: 177.  A stream of the 4-bit pool: 256
// threads with 4 vectors 64 us, 512 with 2: 58, 512 with 1: 69.)
template <int ROW>   // bytes of a key (or value): 256, 128, 64
struct Plain {
  static constexpr int kVecs = 2 * ROW / 16;
  static constexpr int kTail = 0;
  static constexpr int kMovers = 256, kPer = 4, kSteps = 4, kCtas = 3, kSpread = 2;
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
  static constexpr int kMovers = 512, kPer = 2, kSteps = 4, kCtas = 2, kSpread = 1;
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
  static constexpr int kThreads = Row::kMovers, kPer = Row::kPer, kSteps = Row::kSteps;
  static constexpr int kRows = kThreads * kPer / Row::kVecs;   // of a CTA in a step
  static constexpr int kOffTail = kThreads * kPer * 16;
  static constexpr int kOffSum = kOffTail + kRows * 2 * Row::kTail;
  static constexpr int kStepBytes = (kOffSum + kRows * 4 + 15) / 16 * 16;
  static constexpr int kOffMoves = kSteps * kStepBytes;        // lists of kSteps + 1 steps
  static constexpr int kBytes = kOffMoves + (kSteps + 1) * kRows * static_cast<int>(sizeof(Move));
  static constexpr int kKeys = kBytes / 4;                     // ranks that fit it
  // Warps beside the kThreads that move rows: they make the lists.
  static constexpr int kAll = kThreads + kRows;
  static_assert(kRows % 32 == 0, "whole warps, a thread for each row of a step");
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

constexpr uint32_t kStays = 0xffffffffu;   // (above every rank)

struct Shared {
  int hist[2][256];
  __align__(16) int merged[256];
  int counts[3];   // this part's tokens above the threshold, at it; first place that moves
  int warp_counts[2][kMaxWarps];
};

// What stays of a CTA's part [b, e), whose ranks `rank` gives: above a threshold, or at it
// and among the first there.  Writes kept[], and counts[2] of the cluster's CTAs.
template <class Row, class Rank>
__device__ __forceinline__ void select(const EvictArgs& a, cg::cluster_group& cluster, Rank rank,
                                       int b, int e, int want, int32_t* kept, Shared& sh) {
  constexpr int kAll = Ring<Row>::kAll, kWarps = kAll / 32;
  static_assert(kWarps <= kMaxWarps);
  const int C = gridDim.x, c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t prefix = want > 0 ? 0u : kStays - 1;
  int left = want;   // of those that share the prefix
  if (threadIdx.x < 256) sh.hist[0][threadIdx.x] = 0;
  __syncthreads();   // (and the ranks are there)
  if (want > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      int* hist = sh.hist[shift >> 3 & 1 ^ 1];
#pragma unroll 4
      for (int p = b + threadIdx.x; p < e; p += kAll) {
        const uint32_t u = rank(p);
        if (u != kStays && (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8))))
          atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      cluster.sync();
      // (The other histogram was read before this barrier.)
      if (threadIdx.x < 256) {
        int n = 0;
#pragma unroll 8
        for (int k = 0; k < C; ++k) n += cluster.map_shared_rank(hist, k)[threadIdx.x];
        sh.merged[255 - threadIdx.x] = n;
        sh.hist[shift >> 3 & 1][threadIdx.x] = 0;
      }
      __syncthreads();
      // The highest digit at which the counts from above reach `left`, in each warp.
      int n[8];   // digits 255 - 8 lane ... 248 - 8 lane
      *reinterpret_cast<int4*>(n) = reinterpret_cast<const int4*>(sh.merged)[2 * lane];
      *reinterpret_cast<int4*>(n + 4) = reinterpret_cast<const int4*>(sh.merged)[2 * lane + 1];
#pragma unroll
      for (int k = 1; k < 8; ++k) n[k] += n[k - 1];
      int x = n[7];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      int above = x - n[7], digit = 255 - 8 * lane;
      const int short_of = left - above;
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (n[k] < short_of) above = x - n[7] + n[k], digit = 254 - 8 * lane - k;
      const int hit = __ffs(__ballot_sync(0xffffffffu, x >= left)) - 1;
      prefix |= static_cast<uint32_t>(__shfl_sync(0xffffffffu, digit, hit)) << shift;
      left -= __shfl_sync(0xffffffffu, above, hit);
      __syncthreads();   // (merged[] is written again)
    }
  }
  // A warp's share of the part, in whole 32s.
  const int share = ((e - b + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int wb = min(e, b + warp * share), we = min(e, wb + share);
  int before = 0, tied = 0;   // tokens that stay for sure, tied ones: first those of the share
#pragma unroll 4
  for (int p = wb + lane; p < we; p += 32) {
    const uint32_t u = rank(p);
    before += u > prefix;
    tied += u == prefix;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  tied = __reduce_add_sync(0xffffffffu, tied);
  if (lane == 0) sh.warp_counts[0][warp] = before, sh.warp_counts[1][warp] = tied;
  __syncthreads();
  // Then those of the warps before, and, by the first two threads, of the part.
  before = tied = 0;
  int part = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int s0 = sh.warp_counts[0][w], s1 = sh.warp_counts[1][w];
    if (w < warp) before += s0, tied += s1;
    part += threadIdx.x == 0 ? s0 : s1;
  }
  if (threadIdx.x < 3) sh.counts[threadIdx.x] = threadIdx.x < 2 ? part : INT_MAX;
  cluster.sync();
  {
    // And those of the CTAs before.
    int s0 = 0, s1 = 0;
    if (lane < c) {
      const int* other = cluster.map_shared_rank(sh.counts, lane);
      s0 = other[0], s1 = other[1];
    }
    before += __reduce_add_sync(0xffffffffu, s0);
    tied += __reduce_add_sync(0xffffffffu, s1);
  }
  int moved = INT_MAX;   // the first place whose row moves
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int p0 = wb; p0 < we; p0 += 32) {
    const int p = p0 + lane;
    const uint32_t u = p < we ? rank(p) : 0u;
    const bool over = p < we && u > prefix, equal = p < we && u == prefix;
    const unsigned twos = __ballot_sync(0xffffffffu, over), ones = __ballot_sync(0xffffffffu, equal);
    const int t = tied + __popc(ones & below);
    const int j = before + __popc(twos & below) + min(t, left);
    if (over || (equal && t < left)) {
      kept[j] = p;
      if (j != p) moved = min(moved, j);
    }
    before += __popc(twos);
    tied += __popc(ones);
  }
  moved = __reduce_min_sync(0xffffffffu, moved);
  if (lane == 0 && moved != INT_MAX) atomicMin(&sh.counts[2], moved);
  cluster.sync();   // kept[] is complete, and seen by the cluster; the ranks are not needed
}

template <class Row>
__global__ void __launch_bounds__(Ring<Row>::kAll, Row::kCtas)
evict_kernel(const __grid_constant__ EvictArgs a) {
  using R = Ring<Row>;
  constexpr int kThreads = R::kThreads, kPer = R::kPer, kSteps = R::kSteps;
  extern __shared__ __align__(16) uint8_t smem[];   // the part's ranks, then the ring
  __shared__ Shared shared;
  const int kvh = blockIdx.y, i = blockIdx.z;
  const int C = gridDim.x, c = blockIdx.x;   // cluster = grid.x
  const bool mover = threadIdx.x < kThreads;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  // The kernel behind may write the lengths in place: it is let in when this CTA has its
  // own (the branch needs the loaded value).
  const int length = a.seq_lens[i];
  if (length != INT_MIN) pdl_trigger();
  const int seq = max(0, length);
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
  // The ranks of the part are held in shared memory (ones that stay in any case as
  // kStays), or, where they do not fit it, made from the sums each time.
  const int lo = a.first, hi = seq - a.recent, want = a.budget - a.first - a.recent;
  const int per = (seq + C - 1) / C;
  const int b = min(seq, c * per), e = min(seq, b + per);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  auto made = [&](int p) {
    const uint32_t u = rank_of(scores[p]);
    return p < lo || p >= hi ? kStays : u;
  };
  if (per <= R::kKeys) {
#pragma unroll 16
    for (int p = b + threadIdx.x; p < e; p += R::kAll) keys[p - b] = made(p);
    select<Row>(a, cluster, [=](int p) { return keys[p - b]; }, b, e, want, kept, shared);
  } else {
    select<Row>(a, cluster, made, b, e, want, kept, shared);
  }

  // ------------------------------------------------------------ rows
  const int lane = threadIdx.x & 31;
  const int first = lane < C ? cluster.map_shared_rank(shared.counts, lane)[2] : INT_MAX;
  const int from = min(a.budget, __reduce_min_sync(0xffffffffu, first));
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
  auto place = [&](int s, int q) { return from + (s * C + c) * R::kRows + q; };
  // Row q of the list of step s: position p and blocks sb, db for its place j.
  auto put = [&](int s, int q, int j, int p, int sb, int db) {
    Move m{-1, -1, p, 0, 0};
    if (p >= 0) {
      if (sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks) {
        const int so = mod_bs(p, a.bs, a.bs_log2), dof = mod_bs(j, a.bs, a.bs_log2);
        m.from = Row::row(a, sb, so, kvh);
        m.to = Row::row(a, db, dof, kvh);
        m.from_tail = static_cast<int16_t>(Row::tail(so));
        m.to_tail = static_cast<int16_t>(Row::tail(dof));
      } else {
        record_error(a.err, PA_DEVERR_BLOCK_ID);
      }
    }
    moves[s % (kSteps + 1) * R::kRows + q] = m;
  };
  auto position = [&](int s, int j) { return s < steps && j < a.budget ? kept[j] : -1; };
  auto block_of = [&](int p) { return p >= 0 ? table[div_bs(p, a.bs, a.bs_log2)] : -1; };
  int p1 = -1;                      // of the step after the next to be listed
  int p2 = -1, sb = -1, db = -1;    // of the next
  auto list = [&](int s) {          // the list of step s, blocks of s + 1, positions of s + 2
    put(s, q0, place(s, q0), p2, sb, db);
    p2 = p1;
    sb = block_of(p2);
    db = block_of(p2 >= 0 ? place(s + 1, q0) : -1);
    p1 = position(s + 2, place(s + 2, q0));
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
  // The first lists are made by all threads.
#pragma unroll 1
  for (int x = threadIdx.x; x < kSteps * R::kRows; x += R::kAll) {
    const int s = x / R::kRows, q = x % R::kRows, j = place(s, q);
    const int p = position(s, j);
    put(s, q, j, p, block_of(p), block_of(p >= 0 ? j : -1));
  }
  if (!mover) {
    p2 = position(kSteps, place(kSteps, q0));
    p1 = position(kSteps + 1, place(kSteps + 1, q0));
    sb = block_of(p2);
    db = block_of(p2 >= 0 ? place(kSteps, q0) : -1);
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
  // No wait here: this kernel starts when every CTA of the first has read its length and
  // needs nothing else of it (what was before has ended when those run).
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
  // It ends when the first kernel has: what follows in the stream waits for both.
  pdl_trigger();
  pdl_wait();
}

// CTAs for each (request, kv head): as many as let all clusters run at once with kSpread
// CTAs on an SM (a cluster's CTAs share one of the GPU's groups of SMs, which are not
// alike: what fits is asked once for each device), and none with fewer than kLeastRows of
// the budget; kSpread where the clusters are more than that.  One stream of 131072 tokens
// in a 4-bit pool, 8 heads: 12 CTAs 58 us, 8: 70, 16 (7 clusters fit): 68.  128 heads of
// 4096 tokens: 1 CTA 39 us, 2: 40, 4: 54, in bf16 1: 80, 2: 69, 4: 90; 512 heads: 111,
// 125, 175 and 283, 245, 241.
constexpr int kLeastRows = 128;
template <class Row>
int cluster_size(long long units, int budget) {
  static std::mutex mu;
  static bool known[64] = {};
  static int fit[64][kMaxCtas + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    known[dev] = true;
    // Shared memory that kSpread CTAs of an SM have at most.
    constexpr int kShare = 224 * 1024 / Row::kSpread - 8 * 1024;
    static_assert(kShare >= Ring<Row>::kBytes);
    bool ok = cudaFuncSetAttribute(evict_kernel<Row>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kShare) == cudaSuccess;
    const bool wide = ok && cudaFuncSetAttribute(evict_kernel<Row>,
                                                 cudaFuncAttributeNonPortableClusterSizeAllowed,
                                                 1) == cudaSuccess;
    for (int C = 1; ok && C <= (wide ? kMaxCtas : 8); ++C) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(C);
      cfg.blockDim = dim3(Ring<Row>::kAll);
      cfg.dynamicSmemBytes = kShare;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = C;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      ok = cudaOccupancyMaxActiveClusters(&fit[dev][C], evict_kernel<Row>, &cfg) == cudaSuccess;
      if (!ok) fit[dev][C] = 0;
    }
    if (!ok || !wide) cudaGetLastError();   // (a refused size is no error of the call)
  }
  const int most = std::max(1, std::min(kMaxCtas, budget / kLeastRows));
  for (int C = most; C > 1; --C)
    if (fit[dev][C] >= units) return C;
  return fit[dev][1] >= units ? 1 : std::min(most, Row::kSpread);
}

template <class Row>
cudaError_t launch_rows(const EvictArgs& a, int N, cudaStream_t stream) {
  static DeviceFlags smem_set;
  cudaError_t e = set_smem_once(evict_kernel<Row>, Ring<Row>::kBytes, smem_set);
  if (e != cudaSuccess) return e;
  const int C = cluster_size<Row>(static_cast<long long>(N) * a.Hkv, a.budget);
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
    e = n.d == 128 ? launch_rows<Four<128>>(a, n.N, stream)
                   : launch_rows<Four<64>>(a, n.N, stream);
  else if (n.row_bytes == 256)
    e = launch_rows<Plain<256>>(a, n.N, stream);
  else if (n.row_bytes == 128)
    e = launch_rows<Plain<128>>(a, n.N, stream);
  else
    e = launch_rows<Plain<64>>(a, n.N, stream);
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
