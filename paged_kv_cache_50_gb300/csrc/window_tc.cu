// Varlen paged attention with a causal sliding window and first tokens that
// stay visible, on the 5th-generation tensor cores: row j at position p_j sees
// p <= p_j with p > p_j - window or p < sinks; O = softmax(Q K^T scale + M) V
// with the online softmax of "Chapter 1: attention backends", section 4.1.
//
// The tiling is varlen_tc.cu's: a unit is 2 x 128 packed rows (query row, q
// head of a kv group) of one (request, kv head); per 128-token K/V tile S_x =
// Q_x K^T into TMEM, softmax in registers (one row per thread), P back into
// TMEM, O_x += P_x V.  What differs follows from a window's units being short
// (window 1024: nine tiles of ~2 us each, against ~7 us that a CTA takes to
// start, fetch its first operands and drain):
//  * CTAs are persistent.  A running CTA takes over the units of CTAs that
//    were not launched yet (cluster launch control), so the balance is the
//    hardware's and no counter is shared between calls; TMEM, barriers and
//    warps stay.
//  * The units' tiles form one stream.  Tiles, barriers and rings are counted
//    through; the K/V producer and the MMA warp run on into the next unit while
//    the softmax warps still write the last one's output, and the next unit's
//    queries are fetched by TMA as soon as its predecessor's last S has been
//    computed.
//  * A unit's visible context is a list of 16-token pieces: those of the first
//    tokens, then those from its oldest visible position rounded down to 16
//    (one run from position 0 where the two meet).  A tile is eight pieces of
//    the list, so first tokens cost one piece each 16 instead of a tile, and
//    pieces that no row sees are neither read nor looked up.
//  * A piece's keys come in one TMA box (as its values do), both 64-column
//    halves interleaved by 8-row groups.
//
//  * Code is kept short.  Unrolled over a tile's 128 columns, with masks,
//    rescaling and output inline, the hot loops did not fit the SM's
//    instruction cache and the GPC's second level ran at 86 % of its rate (364
//    us on the batch below).  So each row's maximum comes with the TMEM load
//    itself (tcgen05.ld.red), weights are made 32 columns at a time in a loop
//    that reads S again, and masks are written back into S beforehand.
//  * The MMA thread's instructions bound the tile rate next: descriptors are
//    formed by one addition each, and the thread is chosen by elect.sync, so
//    that they live in uniform registers.
//
//  * The grid has one slot per 2 x 128 rows of the whole batch and request, not
//    per request and longest query, and the heads of a slot run side by side (they
//    read neighbouring parts of the same cache rows).
//
// Bound by the chain S -> softmax -> PV -> S of a Q tile (~3200 cycles of a
// 128-token tile pair; its MMAs take 2290) and, at a unit's ends, by mask and
// output code that is not in the instruction cache.  Measured (d 128, 16 requests
// of U[256, 2048] new tokens, 32 / 8 heads, window 1024, 4 first tokens): the
// kernel 275-280 us, 1055-1074 TFLOP/s, a call 283-287; 8192 tokens of 64 / 8
// heads, window 4096: 757-778 us, 1417-1457 TFLOP/s, a call 770;
// varlen_tc.cu's kernel with the same mask, one unit per CTA and 128-token steps,
// took 419 and 1016.  Steps: persistent CTAs 365 / 953; the short loops 318 / 880;
// descriptors 301 / 818; elect.sync 286 / 778; heads side by side 277 / 768.  Two
// MMA threads (368 / 1008), the next unit's first S between the last PVs (328 /
// 915), one loop for all S (354 / 1012) and the weights' next word loaded ahead
// (282 / 790 against 277 / 762) were slower.
//
// Warp roles (384 threads): warp 0 MMA issue; warp 1 K/V producer (lane p:
// piece p); warp 2 units and queries; warp 3 idle; warps 4-7 / 8-11 softmax and
// output of Q tile 0 / 1.  Every wait is bounded; a CTA whose wait runs out sets
// PA_DEVERR_TIMEOUT, stops taking units and leaves.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>
#include <climits>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "tc_tiles.cuh"

namespace pa {

namespace {

template <int D>
struct WinCfg {
  static constexpr int kBM = 128;                    // rows per Q tile
  static constexpr int kBN = 128;                    // tokens per K/V tile
  static constexpr int kPieces = kBN / 16;
  static constexpr int kHalves = D / 64;             // 128-byte column groups of a row
  static constexpr int kQBytes = kBM * D * 2;
  static constexpr int kTileBytes = kBN * D * 2;     // K or V
  static constexpr int kPieceBytes = 16 * D * 2;
  static constexpr int kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffBar = kOffV + 2 * kTileBytes;
  static constexpr int kSmemBytes = kOffBar + 512 + 1024;   // control block + alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 384;
  __host__ __device__ static constexpr uint32_t col_s(int x) { return 128u * x; }
  __host__ __device__ static constexpr uint32_t col_o(int x) { return 256u + 128u * x; }
};

// Barriers; pairs are indexed by stage (tile & 1), unit & 1, or Q tile x.
enum WinBar {
  kQFull = 0,     // [x] queries of the unit have landed
  kQEmpty = 2,    // [x] the unit's last S_x has been computed
  kKFull = 4,
  kKEmpty = 6,
  kVFull = 8,
  kVEmpty = 10,
  kSFull = 12,    // [x]
  kPLo = 14,      // [x] P of tokens 0-95 written
  kPHi = 16,      // [x] P of tokens 96-127 written
  kODone = 18,    // [x] the unit's last PV_x has been computed
  kUnitFull = 20, // [unit & 1] unit descriptor written
  kUnitEmpty = 22,// [unit & 1] ... read by everyone
  kClc = 24,      // response of the launch control
  kFinal = 25,
  kNumBars = 26
};
// Readers of a unit descriptor: MMA, producer, eight softmax warps.
constexpr uint32_t kUnitReaders = 10;

// Control block behind the barriers: byte offsets.
constexpr int kOffTmem = 8 * kNumBars;        // TMEM base (4)
constexpr int kOffAbort = kOffTmem + 4;       // abort flag (4)
constexpr int kOffClc = 224;                  // response (16, 16-byte aligned)
constexpr int kOffRing = 240;                 // loaded-piece masks of four tiles (16)
constexpr int kOffUnits = 256;                // two descriptors
constexpr int kPieceRing = 4;
constexpr int kEmptySlots = 256;   // about half a millisecond

// What a unit is (in shared memory, 64 bytes each).
struct Unit {
  int live;       // 0: no more units
  int request, kvh, q0;
  int rows, tile;   // query rows of the request, and which two Q tiles of them
  int seq, ctx;
  // The unit sees [oldest, end) and the first tokens: `first` pieces from
  // position 0, then pieces from `base`.
  int first, oldest, base, end, pieces, tiles;
};
static_assert(sizeof(Unit) <= 64 && kOffUnits + 2 * 64 <= 512 && kOffAbort + 4 <= kOffClc,
              "layout");

struct WinArgs {
  const int32_t* block_table;
  const int32_t* qsl;
  const int32_t* seq_lens;
  int N, max_blocks, Hq, Hkv, grp, bs, bs_log2, num_blocks;
  int row_tokens;   // query rows of a Q tile: 128 / grp
  int hkv_log2, per_log2;   // of Hkv and 2 * row_tokens where powers of two, else -1
  int total_q, max_query_len;
  int positions;    // of a table row, at most INT_MAX - 127
  float scale_log2;
  int window, sinks;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// 32 consecutive fp32 columns of this thread's TMEM lane and their maximum
// (warp-collective).
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t (&r)[32], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=f"(mx)
      : "r"(taddr));
}

// Whether a phase has completed, without waiting (try_wait may suspend).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// D[tmem] (+)= A B with descriptors given as their low words and a common high
// word each (bits 32-63: stride offset, version, swizzle).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                       uint32_t b_hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.b32 p, %6, 0;\n"
      "mov.b64 da, {%1, %2};\nmov.b64 db, {%3, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 db;\nsetp.ne.b32 p, %5, 0;\nmov.b64 db, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
template <int K>
using Step = std::integral_constant<int, K>;   // a 16-token step of a tile
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(p));
  return p != 0;
}

// Asks for the launch of one more CTA to be cancelled in favour of this one;
// the answer (16 bytes) completes `bar`.
__device__ __forceinline__ void clc_request(uint32_t resp, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(resp),
      "r"(bar)
      : "memory");
}
// Whether a launch was cancelled, and the index of its CTA (of a 1-D grid).
__device__ __forceinline__ bool clc_answer(uint32_t resp, int& x) {
  uint32_t ok;
  asm volatile(
      "{\n"
      ".reg .b128 r;\n"
      ".reg .pred p;\n"
      "ld.shared.b128 r, [%2];\n"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "mov.u32 %1, 0;\n"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n"
      "}\n"
      : "=r"(ok), "=r"(x)
      : "r"(resp)
      : "memory");
  return ok != 0;
}

#ifdef PA_TEST_HOOKS
// Test builds only: the producer of the CTA with index g_window_skip.x issues
// neither the copies nor the byte count of the K of tile g_window_skip.y, so
// the waits on it can only end at their poll limit; {-1, -1} = off.
__device__ int2 g_window_skip = {-1, -1};
// The softmax of Q tile 1 in the CTA with index g_window_mute.x does not publish
// its weights of tile g_window_mute.y (of the CTA's first unit, the last but one),
// and the next unit's queries for Q tile 0 are fetched only when the wait for Q
// tile 1's place has run out.  g_window_left: query copies that were still on
// their way when the CTA took them for landed.
__device__ int2 g_window_mute = {-1, -1};
__device__ int g_window_left = 0;
#endif

// SKIP: words of a tile without pieces are not looked at.
template <int D, bool SKIP>
__global__ void __launch_bounds__(384, 1)
window_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ WinArgs a) {
  using C = WinCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* ctl = smem_raw + (sbase - raw) + C::kOffBar;
  const uint32_t bars = sbase + C::kOffBar;
  auto BAR = [&](int k) { return bars + 8u * static_cast<uint32_t>(k); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + kOffAbort);
  // Ring of loaded-piece masks: (tile << 8) | mask in slot tile % kPieceRing,
  // written by the producer before the tile's K is issued.
  volatile uint32_t* piece_ring = reinterpret_cast<volatile uint32_t*>(ctl + kOffRing);
  auto unit_slot = [&](int u) {
    return reinterpret_cast<volatile Unit*>(ctl + kOffUnits + 64 * (u & 1));
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(BAR(kQFull + b), 1);
      tc::mbar_init(BAR(kQEmpty + b), 1);
      tc::mbar_init(BAR(kKFull + b), 1);
      tc::mbar_init(BAR(kKEmpty + b), 1);
      tc::mbar_init(BAR(kVFull + b), 1);
      tc::mbar_init(BAR(kVEmpty + b), 1);
      tc::mbar_init(BAR(kSFull + b), 1);
      tc::mbar_init(BAR(kPLo + b), C::kBM);
      tc::mbar_init(BAR(kPHi + b), C::kBM);
      tc::mbar_init(BAR(kODone + b), 1);
      tc::mbar_init(BAR(kUnitFull + b), 1);
      tc::mbar_init(BAR(kUnitEmpty + b), kUnitReaders);
    }
    tc::mbar_init(BAR(kClc), 1);
    tc::mbar_init(BAR(kFinal), 1);
    *abort_flag = 0;
    for (int k = 0; k < kPieceRing; ++k) piece_ring[k] = 0xffffffffu;
    tc::fence_barrier_init();
  }
  if (warp == 0) tc::tmem_alloc(bars + kOffTmem, C::kTmemCols);
  if (warp == 1 && lane == 0) {
    tc::tma_prefetch_desc(&q_map);
    tc::tma_prefetch_desc(&k_map);
    tc::tma_prefetch_desc(&v_map);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(ctl + kOffTmem);
  auto fail = [&]() {
    record_error(a.err, PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  // Inputs and the output buffer may belong to the previous kernel until here.
  pdl_wait();

  if (warp >= 4) {
    // ------------------------------------------------------ softmax, output
    const int x = (warp >> 2) - 1;
    const int t = threadIdx.x & 127;         // row within the tile = TMEM lane
    const int t_tok = t / a.grp, hh = t - t_tok * a.grp;
    const bool row_used = t_tok < a.row_tokens;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::col_s(x), to = tmem + lane_base + C::col_o(x);
    // TMEM loads and stores are warp-collective: every decision to skip or
    // stop is taken for the whole warp.
    auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
      const bool w = __all_sync(0xffffffffu, tc::mbar_wait(b, parity));
      if (!w) fail();
      return w;
    };
    uint32_t g = 0, full = 0;   // tiles and units with tiles so far
    for (int u = 0;; ++u) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      if (!wait_warp(BAR(kUnitFull + (u & 1)), (u >> 1) & 1)) break;
      volatile Unit* un = unit_slot(u);
      const int live = un->live, ntiles = un->tiles, n_first = un->first, tbase = un->base;
      const int end = un->end, oldest = un->oldest;
      const int qi = (un->tile * 2 + x) * a.row_tokens + t_tok;   // query row of the request
      const bool valid = row_used && qi < un->rows;
      const int lim = valid ? max(0, min(un->ctx + qi + 1, un->seq)) : 0;
      const int64_t qrow = static_cast<int64_t>(un->q0 + qi) * a.Hq + un->kvh * a.grp + hh;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR(kUnitEmpty + (u & 1)));
      if (!live) break;
      const int unit_lo = max(0, lim - a.window);
      // l: the row's sum of weights (for the LSE); lr: the same weights rounded
      // to bf16, as PV multiplies them (the output's divisor).
      float m_used = -CUDART_INF_F, l = 0.f, lr = 0.f;
      bool alive = true;
      for (int j = 0; j < ntiles; ++j, ++g) {
        if (__any_sync(0xffffffffu, *abort_flag != 0) || !wait_warp(BAR(kSFull + x), g & 1)) {
          alive = false;
          break;
        }
        tc::tc_fence_after();
        uint32_t vm;
        {
          const uint32_t tag = g << 8;
          uint32_t w = piece_ring[g % kPieceRing];
          for (int n = 0; (w & ~0xffu) != tag && n < tc::kWaitPolls; ++n)
            w = piece_ring[g % kPieceRing];
          if (!__all_sync(0xffffffffu, (w & ~0xffu) == tag)) {
            fail();
            alive = false;
            break;
          }
          vm = w & 0xffu;
        }
        // With SKIP, 32-column words of the tile up to its last loaded piece; the
        // others' weights are zeros.  Formed anew from the mask where it is used: a
        // register less over the maxima.
        auto words = [&]() { return SKIP ? (33 - __clz(vm)) >> 1 : C::kBN / 32; };
        // Position of column 0 as if the tile held no first tokens; mask only
        // where some column is not visible.  (Decided for the whole warp, and
        // done in tensor memory, word by word, so that the code is short.)
        const int tok0 = tbase + j * C::kBN - 16 * n_first;
        // The window's first position (or one below 0; recomputed for a register).
        const int lo = SKIP ? lim - a.window : unit_lo;
        if (__any_sync(0xffffffffu, !(tok0 + C::kBN <= lim && tok0 >= lo && tok0 >= tbase &&
                                      vm == 0xffu))) {
          // Visible columns as bits: the window's range [wa, wb), past the
          // columns of the first tokens' pieces, and the first tokens [0, fe).
          // (Where wb < 0 the window shows nothing, and wb - window could leave 32 bits.)
          const int cf = max(0, min(16 * n_first - j * C::kBN, C::kBN));
          const int wb = lim - tok0, wa = max(max(wb, 0) - a.window, cf);
          const int fe = cf > 0 ? min(cf, min(a.sinks, lim) - j * C::kBN)
                                : min(a.sinks, lim) - tok0;
#pragma unroll 1
          for (int w = 0; w < words(); ++w) {
            const uint32_t loaded = ((vm >> (2 * w)) & 1u ? 0xffffu : 0u) |
                                    ((vm >> (2 * w + 1)) & 1u ? 0xffff0000u : 0u);
            const uint32_t bits = ((bits_below(wb - 32 * w) & ~bits_below(wa - 32 * w)) |
                                   bits_below(fe - 32 * w)) & loaded;
            if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
            uint32_t r[32];
            tc::tmem_ld32(ts + w * 32, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = (bits >> c) & 1u ? r[c] : 0xff800000u;   // -inf
            tc::tmem_st32(ts + w * 32, r);
          }
          tc::tmem_wait_st();
        }
        float mx;
        {
          uint32_t r[C::kBN / 32][32];
          float m4[C::kBN / 32];
#pragma unroll
          for (int c = 0; c < C::kBN / 32; ++c) tmem_ld32_max(ts + c * 32, r[c], m4[c]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < C::kBN / 32; ++c)
            if (c >= words()) m4[c] = -CUDART_INF_F;
          mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
          mx *= a.scale_log2;
        }
        const float m_new = fmaxf(m_used, mx);
        const bool need = m_new > m_used + 8.f;
        const float alpha = need ? ex2(m_used - m_new) : 1.f;
        if (need) m_used = m_new;
        const float mu = m_used == -CUDART_INF_F ? 0.f : m_used;
        // S_x(j) has landed, hence PV_x(j-1) too: O_x may be rescaled now.
        if (__any_sync(0xffffffffu, need) && j > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tc::tmem_ld32(to + c * 32, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tc::tmem_st32(to + c * 32, r);
          }
        }
        // V rows that no query of the unit sees may hold anything (0 * NaN is
        // NaN): cleared once V has landed, one row per thread, by both
        // warpgroups, each before it publishes its own P.
        {
          const int v = j * C::kPieces + (t >> 4);
          const int tok = (v < n_first ? 16 * v : tbase + 16 * (v - n_first)) + (t & 15);
          if (!(tok < end && (tok >= oldest || tok < a.sinks) && ((vm >> (t >> 4)) & 1u))) {
            if (!tc::mbar_wait(BAR(kVFull + (g & 1)), (g >> 1) & 1)) fail();
            const uint32_t vbase = sbase + C::kOffV + (g & 1) * C::kTileBytes +
                                   (t >> 4) * C::kPieceBytes;
#pragma unroll 1
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll 1
              for (int c = 0; c < 8; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vbase + h * 2048 +
                                                                           sw128(t & 15, c)),
                             "r"(0u)
                             : "memory");
            tc::fence_proxy_async_smem();   // before this thread's P arrival
          }
        }
        // P = exp2(s * scale_log2 - m_used) as bf16 pairs over the first 64
        // columns of the S row (behind the columns still to be read), published
        // after 96 and after 128 tokens: what is left of PV_x for the chain is
        // two steps.
        {
          auto publish = [&](int c) {
            tc::tmem_wait_st();
            tc::tc_fence_before();
#ifdef PA_TEST_HOOKS
            if (x == 1 && blockIdx.x == static_cast<unsigned>(g_window_mute.x) &&
                g == static_cast<uint32_t>(g_window_mute.y))
              return;
#endif
            tc::mbar_arrive(BAR((c == 2 ? kPLo : kPHi) + x));
          };
          float l8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          float r8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c = 0; c < words(); ++c) {
            uint32_t r[32], pk[16];
            tc::tmem_ld32(ts + c * 32, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              ffma2(x0, x1, __uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]), a.scale_log2,
                    -mu);
              const float p0 = ex2(x0);
              const float p1 = ex2(x1);
              fadd2(l8[2 * (e & 3)], l8[2 * (e & 3) + 1], p0, p1);
              pk[e] = pack_bf16(p0, p1);
              add_bf16x2_f32(r8[2 * (e & 3)], r8[2 * (e & 3) + 1], pk[e]);
            }
            tc::tmem_st16(ts + c * 16, pk);
            if (c >= 2) publish(c);
          }
#pragma unroll 1
          for (int c = words(); c < C::kBN / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0u;
            tc::tmem_st16(ts + c * 16, pk);
            if (c >= 2) publish(c);
          }
          l = l * alpha +
              (((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7])));
          lr = lr * alpha +
               (((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7])));
        }
      }
      if (alive && ntiles > 0) {
        alive = wait_warp(BAR(kODone + x), full & 1);
        ++full;
      }
      if (alive && ntiles > 0) {   // warp-uniform
        tc::tc_fence_after();
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
        // 32-byte stores write whole sectors where `out` is 32-byte aligned.
        const bool a32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + qrow * D);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          tc::tmem_ld32(to + c * 32, r);
          tc::tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = pack_bf16(__uint_as_float(r[v * 16 + 2 * e]) * inv,
                                 __uint_as_float(r[v * 16 + 2 * e + 1]) * inv);
              uint32_t* p = dst + c * 16 + v * 8;
              if (a32) {
                st_global_v8(p, w);
              } else {
                reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
        if (valid && a.lse != nullptr)
          a.lse[qrow] = l == 0.f ? -CUDART_INF_F : (m_used + log2f(l)) * kLn2;
      } else if (valid) {
        // Nothing visible (or a CTA that gave up): o = 0, lse = -inf.
        uint4* dst = reinterpret_cast<uint4*>(a.out + qrow * D);
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr) a.lse[qrow] = -CUDART_INF_F;
      }
      // The output's TMEM reads come before this warp's next P arrival, which
      // the next unit's first PV waits for.
      tc::tc_fence_before();
      if (!alive) break;
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ MMA issue
    if (elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, C::kBN, 0, 0);
      constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, 0, 1);
      uint32_t g = 0, full = 0;
      bool ok = true;
      auto wait = [&](int bar, uint32_t parity) { return tc::mbar_wait(BAR(bar), parity); };
      // Low words of the descriptors at the buffers' starts (offset 16 for the
      // unused leading dimension of Q and K, 2048 between V's column halves).
      const uint32_t q_lo = (sbase >> 4) | (1u << 16);
      const uint32_t k_lo = ((sbase + C::kOffK) >> 4) | (1u << 16);
      const uint32_t v_lo = ((sbase + C::kOffV) >> 4) | (128u << 16);
      // S_x of tile n (of the stream) into the S columns of tile x.
      auto issue_s = [&](int x, uint32_t n) {
        const uint32_t ql = q_lo + x * (C::kQBytes >> 4);
        const uint32_t kl = k_lo + (n & 1) * (C::kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          // K: [8-row group][half][8 rows][128 B].
          mma_ss(tmem + C::col_s(x), ql + (((k >> 2) * (C::kBM * 128) + (k & 3) * 32) >> 4),
                 desc_hi(1024), kl + (((k >> 2) * 1024 + (k & 3) * 32) >> 4),
                 desc_hi(1024 * C::kHalves), idesc_s, k > 0);
        tc::mma_commit(BAR(kSFull + x));
      };
      // O_x (+)= P_x V over the 16-token steps [from, to).
      auto issue_pv = [&](int x, uint32_t n, auto from, auto to, bool fresh) {
        const uint32_t vl = v_lo + (n & 1) * (C::kTileBytes >> 4);
#pragma unroll
        for (int k = from; k < to; ++k)
          mma_ts(tmem + C::col_o(x), tmem + C::col_s(x) + k * 8, vl + k * (C::kPieceBytes >> 4),
                 desc_hi(1024), idesc_o, !fresh || k > 0);
      };
      for (int u = 0; ok; ++u) {
        if (*abort_flag || !wait(kUnitFull + (u & 1), (u >> 1) & 1)) { ok = false; break; }
        volatile Unit* un = unit_slot(u);
        const int live = un->live, ntiles = un->tiles;
        tc::mbar_arrive(BAR(kUnitEmpty + (u & 1)));
        if (!live) break;
        if (ntiles == 0) continue;
        // First S of both tiles; the queue runs on from the unit before.
        if (!wait(kKFull + (g & 1), (g >> 1) & 1)) { ok = false; break; }
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
          ok = wait(kQFull + x, full & 1);
          if (!ok) break;
          tc::tc_fence_after();
          issue_s(x, g);
          if (ntiles == 1) tc::mma_commit(BAR(kQEmpty + x));
        }
        if (!ok) break;
        tc::mma_commit(BAR(kKEmpty + (g & 1)));
        for (int j = 0; ok && j < ntiles; ++j, ++g) {
          if (*abort_flag) { ok = false; break; }
          const bool more = j + 1 < ntiles;
          if (!wait(kVFull + (g & 1), (g >> 1) & 1)) { ok = false; break; }
          if (more && !wait(kKFull + ((g + 1) & 1), ((g + 1) >> 1) & 1)) { ok = false; break; }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!wait(kPLo + x, g & 1)) { ok = false; break; }
            tc::tc_fence_after();
            issue_pv(x, g, Step<0>(), Step<6>(), j == 0);
            if (!wait(kPHi + x, g & 1)) { ok = false; break; }
            tc::tc_fence_after();
            issue_pv(x, g, Step<6>(), Step<8>(), false);
            if (more) {
              issue_s(x, g + 1);
              if (j + 2 == ntiles) tc::mma_commit(BAR(kQEmpty + x));
            } else {
              tc::mma_commit(BAR(kODone + x));
            }
          }
          if (!ok) break;
          tc::mma_commit(BAR(kVEmpty + (g & 1)));
          if (more) tc::mma_commit(BAR(kKEmpty + ((g + 1) & 1)));
        }
        ++full;
      }
      if (!ok && !*abort_flag) fail();
      // Everything issued has completed before TMEM is released.
      tc::mma_commit(BAR(kFinal));
      if (!tc::mbar_wait(BAR(kFinal), 0)) fail();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ K/V producer
    // Lane p looks after piece p of each tile.  K runs up to two tiles ahead of
    // V, across units: K(g+1), V(g), K(g+2), V(g+1), ...; V reuses its K's block
    // ids.  Block ids are loaded two tiles ahead and validated when used.
    const bool box = lane < C::kPieces;
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity));
    };
    uint32_t gk = 0, gv = 0;          // tiles whose K / V have been issued
    // The lane's pieces in tiles gv and gv + 1: block (-1: not loaded), first
    // token's offset in it, kv head.
    int blk0 = -1, blk1 = -1, off0 = 0, off1 = 0;
    int kvh0 = 0, kvh1 = 0;
    int u = 0, j = 0, ntiles = 0;     // the unit that K is in
    int request = 0, kvh = 0, n_first = 0, tbase = 0, pieces = 0;
    int r0 = -1, r1 = -1;             // raw ids of tiles j, j + 1
    bool ok = true, more = true;      // more: units may follow
    auto raw_of = [&](int jj) -> int {
      const int v = jj * C::kPieces + lane;
      if (!box || v >= pieces) return -1;
      const int idx = div_bs(v < n_first ? 16 * v : tbase + 16 * (v - n_first), a.bs, a.bs_log2);
      // (A plain load: the table may be the previous kernel's output.)
      return idx < a.max_blocks
                 ? a.block_table[static_cast<int64_t>(request) * a.max_blocks + idx] : -1;
    };
    while (ok && (more || gv < gk)) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      bool do_k = more && gk < gv + 2;
      if (do_k && j == ntiles) {
        // The next unit; with a V outstanding, only if it is known already.
        const uint32_t bar = BAR(kUnitFull + (u & 1)), parity = (u >> 1) & 1;
        const bool known = gv < gk ? __all_sync(0xffffffffu, mbar_test(bar, parity))
                                   : wait_all(bar, parity);
        if (!known && gv == gk) { ok = false; break; }
        do_k = false;
        if (known) {
          volatile Unit* un = unit_slot(u);
          more = un->live != 0;
          request = un->request;
          kvh = un->kvh;
          n_first = un->first;
          tbase = un->base;
          pieces = un->pieces;
          ntiles = un->tiles;
          j = 0;
          ++u;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(BAR(kUnitEmpty + ((u - 1) & 1)));
          if (!more) ntiles = 0;
          r0 = ntiles > 0 ? raw_of(0) : -1;
          r1 = ntiles > 1 ? raw_of(1) : -1;
          continue;
        }
      }
      if (do_k) {
        const int st = gk & 1;
        const int r2 = j + 2 < ntiles ? raw_of(j + 2) : -1;
        if (gk >= 2 && !wait_all(BAR(kKEmpty + st), ((gk >> 1) - 1) & 1)) { ok = false; break; }
        const int v = j * C::kPieces + lane;
        const bool mine = box && v < pieces;
#ifdef PA_TEST_HOOKS
        const bool skip = blockIdx.x == static_cast<unsigned>(g_window_skip.x) &&
                          gk == static_cast<uint32_t>(g_window_skip.y);
#else
        constexpr bool skip = false;
#endif
        const bool good = mine && r0 >= 0 && r0 < a.num_blocks && !skip;
        const int blk = good ? r0 : -1;
        const int off = mod_bs(v < n_first ? 16 * v : tbase + 16 * (v - n_first), a.bs, a.bs_log2);
        const unsigned loaded = __ballot_sync(0xffffffffu, good);
        const unsigned bad = __ballot_sync(0xffffffffu, mine && !good);
        if (lane == 0) {
          if (bad != 0u && !skip) record_error(a.err, PA_DEVERR_BLOCK_ID);
          piece_ring[gk % kPieceRing] = (gk << 8) | (loaded & 0xffu);
          if (!skip)
            tc::mbar_arrive_expect_tx(BAR(kKFull + st),
                                      static_cast<uint32_t>(__popc(loaded)) * C::kPieceBytes);
        }
        __syncwarp();
        // Coordinates: column, token in its 8-group, half (of all heads'), token
        // group, 2 * block.
        if (good)
          tc::tma_load_5d(sbase + C::kOffK + st * C::kTileBytes + lane * C::kPieceBytes, &k_map,
                          BAR(kKFull + st), 0, 0, kvh * C::kHalves, off >> 3, 2 * blk);
        if (gk == gv) {
          blk0 = blk, off0 = off, kvh0 = kvh;
        } else {
          blk1 = blk, off1 = off, kvh1 = kvh;
        }
        r0 = r1;
        r1 = r2;
        ++j;
        ++gk;
      } else if (gv < gk) {
        const int st = gv & 1;
        if (gv >= 2 && !wait_all(BAR(kVEmpty + st), ((gv >> 1) - 1) & 1)) { ok = false; break; }
        const unsigned loaded = __ballot_sync(0xffffffffu, blk0 >= 0);
        if (lane == 0)
          tc::mbar_arrive_expect_tx(BAR(kVFull + st),
                                    static_cast<uint32_t>(__popc(loaded)) * C::kPieceBytes);
        __syncwarp();
        if (blk0 >= 0)
          tc::tma_load_5d(sbase + C::kOffV + st * C::kTileBytes + lane * C::kPieceBytes, &v_map,
                          BAR(kVFull + st), 0, off0, 0, kvh0, 2 * blk0 + 1);
        blk0 = blk1, off0 = off1, kvh0 = kvh1;
        ++gv;
      }
    }
    if (lane == 0) {
      if (!ok) fail();
      // No copy may still be landing when the CTA exits.
      for (uint32_t n = gk >= 2 ? gk - 2 : 0; n < gk; ++n)
        if (!tc::mbar_wait(BAR(kKFull + (n & 1)), (n >> 1) & 1)) fail();
      for (uint32_t n = gv >= 2 ? gv - 2 : 0; n < gv; ++n)
        if (!tc::mbar_wait(BAR(kVFull + (n & 1)), (n >> 1) & 1)) fail();
    }
  } else if (warp == 2) {
    // ------------------------------------------------------ units and queries
    // Slot s of the grid belongs to the last request i with qsl[i] / per + i <=
    // s (per: query rows of a unit): request i owns at least ceil(qlen / per)
    // slots from there on, and the grid has total_q / per + N slots, so that a
    // batch of many short and a few long requests has at most one empty slot
    // per request.  The request is found by a 32-way search.
    // The heads of a slot run side by side: they read neighbouring parts of the
    // same cache rows and queries.
    int slot = div_bs(blockIdx.x, a.Hkv, a.hkv_log2), head = blockIdx.x - slot * a.Hkv;
    const int per = 2 * a.row_tokens;
    const uint32_t resp = bars + kOffClc;
    bool ok = true, asked = false;
    uint32_t answers = 0, full = 0, fetched = 0;   // fetched: Q tiles, 0 and 1 in turn
    int empty = 0;   // empty slots in a row
    // Unlike the others, these waits last as long as a unit.
    auto wait = [&](int bar, uint32_t parity) {
      for (int n = 0; n < 64; ++n) {
        if (tc::mbar_wait(BAR(bar), parity)) return true;
        if (*abort_flag) return false;
      }
      return false;
    };
    auto ask = [&]() {
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(BAR(kClc), 16);
        clc_request(resp, BAR(kClc));
      }
      asked = true;
    };
    ask();
    int u = 0;
    for (bool live = true; live;) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
      int lo = 0, hi = a.N, q0 = 0, q1 = 0, seq = 0;
      for (;;) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool in = i < hi;
        const int q = in ? a.qsl[i] : 0;
        const bool last = step == 1;
        // In the last round a lane holds its request's row.
        const int next = in && last ? a.qsl[i + 1] : 0;
        const int len = in && last ? a.seq_lens[i] : 0;
        const unsigned below = __ballot_sync(0xffffffffu, in && div_bs(q, per, a.per_log2) + i <= slot);
        const int k = max(31 - __clz(below), 0);
        lo += k * step;
        hi = min(lo + step, hi);
        if (last) {
          q0 = __shfl_sync(0xffffffffu, q, k);
          q1 = __shfl_sync(0xffffffffu, next, k);
          seq = max(0, __shfl_sync(0xffffffffu, len, k));
          break;
        }
      }
      const int qlen = q1 - q0, tile = slot - (div_bs(q0, per, a.per_log2) + lo), qi = tile * per;   // first query row
      // Rows past max_query_len, or outside the batch, are not touched.
      const int rows = q0 >= 0 ? min(min(qlen, a.max_query_len), a.total_q - q0) : 0;
      const bool real = tile >= 0 && qi < rows;
      // A long run of empty slots is broken by units without rows, so that the
      // other warps' waits for a unit stay short.
      empty = real ? 0 : empty + 1;
      if (real || empty == kEmptySlots) {
        empty = 0;
        const int ctx = seq - qlen;
        const int q_last = min(qi + per, rows) - 1;
        // Positions [0, end) and, in the window, from `oldest` on; what lies past
        // the table's columns has no block and is not walked over.
        int end = max(0, min(ctx + q_last + 1, seq));
        if (real && end > a.positions) {
          if (lane == 0) record_error(a.err, PA_DEVERR_BLOCK_ID);
          end = a.positions;
        }
        // (A first row before position 0 is held to 0 before the window is taken
        // off: the difference fits an int whatever the window.)
        const int oldest = max(0, max(0, ctx + qi + 1) - a.window);
        int first = (min(a.sinks, end) + 15) >> 4, base = oldest & ~15;
        if (base <= 16 * first) first = base = 0;
        const int pieces = first + ((max(0, end - base) + 15) >> 4);
        const int tiles = real ? (pieces + C::kPieces - 1) / C::kPieces : 0;
        if (u >= 2 &&
            !__all_sync(0xffffffffu, wait(kUnitEmpty + (u & 1), ((u >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          volatile Unit* un = unit_slot(u);
          un->live = 1;
          un->request = lo;
          un->kvh = head;
          un->q0 = q0;
          un->rows = real ? rows : 0;
          un->tile = tile;
          un->seq = seq;
          un->ctx = ctx;
          un->first = first;
          un->oldest = oldest;
          un->base = base;
          un->end = end;
          un->pieces = pieces;
          un->tiles = tiles;
          tc::mbar_arrive(BAR(kUnitFull + (u & 1)));
        }
        __syncwarp();
        ++u;
        if (tiles > 0) {
          // Rows past the request or the batch are fetched too (or zeros): they are
          // masked.
          auto fetch = [&](int x) {
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(
                  BAR(kQFull + x), static_cast<uint32_t>(a.row_tokens * a.grp) * (D * 2));
              for (int h = 0; h < C::kHalves; ++h)
                tc::tma_load_3d(sbase + x * C::kQBytes + h * (C::kBM * 128), &q_map,
                                BAR(kQFull + x), h * 64, head * a.grp,
                                min(q0 + qi + x * a.row_tokens, a.total_q));
            }
          };
#ifdef PA_TEST_HOOKS
          const bool late = full == 1 && blockIdx.x == static_cast<unsigned>(g_window_mute.x);
#else
          constexpr bool late = false;
#endif
          for (int x = 0; x < 2 && ok; ++x) {
            if (full > 0 &&
                !__all_sync(0xffffffffu, wait(kQEmpty + x, (full - 1) & 1))) {
              if (late && x == 1) fetch(0);
              ok = false;
              break;
            }
            if (!late) fetch(x);
            ++fetched;
          }
          if (!ok) break;
          ++full;
        }
      }
      // The next unit, if a launch is left to take over.
      if (!__all_sync(0xffffffffu, wait(kClc, answers & 1))) {
        ok = false;
        break;
      }
      ++answers;
      asked = false;
      int cta;
      live = clc_answer(resp, cta);
      slot = div_bs(cta, a.Hkv, a.hkv_log2);
      head = cta - slot * a.Hkv;
      if (live) {
        tc::fence_proxy_async_smem();   // the answer has been read
        __syncwarp();
        ask();
      }
    }
    if (ok && u >= 2)
      ok = __all_sync(0xffffffffu, wait(kUnitEmpty + (u & 1), ((u >> 1) - 1) & 1));
    if (lane == 0) {
      if (ok) {
        unit_slot(u)->live = 0;
        unit_slot(u)->tiles = 0;
        tc::mbar_arrive(BAR(kUnitFull + (u & 1)));
      } else {
        fail();
      }
      // Nothing may land in shared memory any more.
      if (asked) tc::mbar_wait(BAR(kClc), answers & 1);
      // (A unit may have been given up between its two Q tiles.)
      for (int x = 0; x < 2; ++x) {
        const uint32_t n = (fetched + 1 - x) >> 1;
        if (n > 0) tc::mbar_wait(BAR(kQFull + x), (n - 1) & 1);
      }
#ifdef PA_TEST_HOOKS
      for (uint32_t n = fetched >= 2 ? fetched - 2 : 0; n < fetched; ++n)
        if (!mbar_test(BAR(kQFull + (n & 1)), (n >> 1) & 1)) atomicAdd(&g_window_left, 1);
#endif
    }
  }

  pdl_trigger();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

// Queries [T][Hq][d]: 64 columns x the heads of a group x the query rows of a
// Q tile.
bool make_q_map(CUtensorMap* map, const void* q, int T, int Hq, int d, int grp, int row_tokens) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t strides[2] = {row, row * Hq};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(grp), static_cast<cuuint32_t>(row_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys so that one box holds a 16-token piece as [8-row group][half][8 rows][128
// B]: dims (innermost first) 64 columns, 8 tokens, d/64 * Hkv halves, bs/8
// groups, 2 nb (2 * block); box 64 x 8 x d/64 x 2 x 1.
bool make_k_map(CUtensorMap* map, const void* cache, int nb, int bs, int Hkv, int d) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(Hkv) * (d / 64),
                              static_cast<cuuint64_t>(bs / 8), 2 * static_cast<cuuint64_t>(nb)};
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t strides[4] = {row * Hkv, 128, row * Hkv * 8, row * Hkv * bs};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d / 64), 2, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SKIP>
cudaError_t launch_t(const WindowPrefillLaunch& n, cudaStream_t stream) {
  using C = WinCfg<D>;
  WinArgs a{};
  a.block_table = n.block_table;
  a.qsl = n.qsl;
  a.seq_lens = n.seq_lens;
  a.max_blocks = n.max_blocks;
  a.Hq = n.Hq;
  a.N = n.N;
  a.Hkv = n.Hkv;
  a.grp = n.Hq / n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  a.num_blocks = n.num_blocks;
  a.row_tokens = C::kBM / a.grp;
  a.hkv_log2 = block_size_log2(n.Hkv);
  a.per_log2 = block_size_log2(2 * a.row_tokens);
  a.total_q = n.total_q;
  a.max_query_len = n.max_query_len;
  a.positions = static_cast<int>(
      std::min(static_cast<long long>(n.max_blocks) * n.bs, INT_MAX - 127LL));
  a.scale_log2 = n.scale * kLog2e;
  a.window = n.window;
  a.sinks = n.sinks;
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  CUtensorMap q_map, k_map, v_map;
  // TMA coordinates are 32-bit.
  if (2LL * n.num_blocks > INT_MAX ||
      !make_q_map(&q_map, n.q, n.total_q, n.Hq, D, a.grp, a.row_tokens) ||
      !make_k_map(&k_map, n.cache, n.num_blocks, n.bs, n.Hkv, D) ||
      !make_v_map(&v_map, n.cache, n.num_blocks, n.bs, n.Hkv, D))
    return cudaErrorInvalidValue;
  auto kern = window_tc_kernel<D, SKIP>;
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  // Slots of the grid, per head: see the scheduler.
  const long long ctas = (n.total_q / (2 * a.row_tokens) + static_cast<long long>(n.N)) * n.Hkv;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(C::kThreads), C::kSmemBytes,
                    stream, q_map, k_map, v_map, a);
}

}  // namespace

#ifdef PA_TEST_HOOKS
// Test builds only (not declared in pa.h).
extern "C" int pa_test_skip_window_tile(int cta, int tile) {
  const int2 v = make_int2(cta, tile);
  return cudaMemcpyToSymbol(g_window_skip, &v, sizeof(v)) == cudaSuccess ? 0 : 3;
}
extern "C" int pa_test_mute_window_tile(int cta, int tile) {
  const int2 v = make_int2(cta, tile);
  return cudaMemcpyToSymbol(g_window_mute, &v, sizeof(v)) == cudaSuccess ? 0 : 3;
}
// What g_window_left has counted since the last call.
extern "C" int pa_test_window_left(int* copies) {
  const int none = 0;
  return cudaMemcpyFromSymbol(copies, g_window_left, sizeof(none)) == cudaSuccess &&
                 cudaMemcpyToSymbol(g_window_left, &none, sizeof(none)) == cudaSuccess
             ? 0 : 3;
}
#endif

cudaError_t launch_window_prefill(const WindowPrefillLaunch& n, cudaStream_t stream) {
  if (n.d == 64) return launch_t<64, true>(n, stream);
  // Where a unit sees a few tiles only, those that end early are many, and their
  // empty words are worth skipping, which costs a full tile 1.5 % (us with and
  // without, d 128: three requests of at most 5 tokens 5.2, 6.2; windows of 64 110,
  // 121, 192 138, 146, 384 164.6, 164.6, 512 189.0, 188.2, 1024 281, 277; d 64: 128 165,
  // 186, 1024 469, 473).
  const long long seen = std::min(static_cast<long long>(n.window) + n.sinks,
                                  static_cast<long long>(n.max_blocks) * n.bs);
  return seen <= 384 ? launch_t<128, true>(n, stream) : launch_t<128, false>(n, stream);
}

}  // namespace pa
