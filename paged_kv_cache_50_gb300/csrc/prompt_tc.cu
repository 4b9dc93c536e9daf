// Causal attention over whole prompts on the 5th-generation tensor cores: queries,
// keys and values of several prompts packed one after another, row j of a prompt sees
// its rows <= j; O = softmax(scale Q K^T + M) V with the online softmax of "Chapter 1:
// attention backends", section 4.1.  Nothing goes through a block pool: the keys and
// values are the step's own, wherever the projection (or a rotation) left them.
//
// The frame is window_tc.cu's: persistent CTAs that take over each other's units by
// cluster launch control, units of 2 x 128 packed rows (query row, q head of a kv
// group), a stream of 128-token K/V tiles counted through from unit to unit, S and P in
// TMEM, next queries fetched as soon as the last S is done.  What differs:
//  * K and V come by plain TMA tiles (128 tokens x 64 columns), each by a thread of
//    its own, with nothing to look up.
//  * Four softmax warpgroups instead of two: each Q tile's rows are halved by columns
//    (tokens 0-63 and 64-127 of a tile).  A tile pair's MMAs take ~2200 cycles, and what
//    a Q tile's softmax takes between its S and its P must pass within half of that,
//    while the other Q tile's MMAs run; one thread per row needs about twice that.
//    The halves exchange their maxima through shared memory (a barrier of two warps)
//    and else work apart: each writes its P over its own S columns and rescales and
//    stores its half of O.  The weights' sums are formed once P is published, while the
//    MMAs run (between S and P: 820 us for a prompt of 8192 tokens, so 775).
//  * Units go longest first: a unit's work grows with its place in the prompt.
//    With up to 64 prompts the order runs over all of them, else within each.
//
// Bound by the chain S -> softmax -> PV of a Q tile, ~3000 cycles for a tile pair, in which
// 16 warps issue ~8000 instructions; and by units' ends (6 tiles each for 16 prompts of up
// to 2048 tokens).  One prompt of 8192 tokens, 64 heads of 128: 742 us, 1.48 PFLOP/s; the 16
// prompts, 32 heads: 202 us, 1.06.
//
// Warp roles (640 threads): warp 0 MMA issue; warp 1 K; warp 2 units and queries; warp
// 3 V; warps 4-7, 8-11 halves 0, 1 of Q tile 0; warps 12-15, 16-19 of Q tile 1.  Every
// wait is bounded; a CTA whose wait runs out sets PA_DEVERR_TIMEOUT and leaves.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "pa_common.cuh"
#include "pa_launch.h"
#include "tc_issue.cuh"
#include "tc_tiles.cuh"

namespace pa {

namespace {

template <int D>
struct PromptCfg {
  static constexpr int kBM = 128;                    // rows per Q tile
  static constexpr int kBN = 128;                    // tokens per K/V tile
  static constexpr int kHalves = D / 64;             // 128-byte column groups of a row
  static constexpr int kQBytes = kBM * D * 2;
  static constexpr int kTileBytes = kBN * D * 2;     // K or V
  static constexpr int kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffBar = kOffV + 2 * kTileBytes;
  static constexpr int kOffMax = kOffBar + 1024;     // [tile & 1][x][half][128] floats
  static constexpr int kOffSum = kOffMax + 4096;     // [x][half][128] float2
  static constexpr int kOffRows = kOffSum + 4096;    // [128] query row within the tile, head
  static constexpr int kSmemBytes = kOffRows + 1024 + 1024;   // + alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 640;
  static constexpr uint32_t kRegSoftmax = 104;
  static constexpr uint32_t kRegOther = 64;
  __host__ __device__ static constexpr uint32_t col_s(int x) { return 128u * x; }
  __host__ __device__ static constexpr uint32_t col_o(int x) { return 256u + 128u * x; }
};

// Barriers; pairs are indexed by stage (tile & 1), unit & 1, or Q tile x.
enum PromptBar {
  kQFull = 0,      // [x] queries of the unit have landed
  kQEmpty = 2,     // [x] the unit's last S_x has been computed
  kKFull = 4,
  kKEmpty = 6,
  kVFull = 8,
  kVEmpty = 10,
  kSFull = 12,     // [x]
  kPLo = 14,       // [x] P of tokens 0-31 and 64-95 written
  kPHi = 16,       // [x] ... and of the others
  kODone = 18,     // [x] the unit's last PV_x has been computed
  kUnitFull = 20,  // [unit & 1]
  kUnitEmpty = 22, // [unit & 1]
  kClc = 24,
  kFinal = 25,
  kPair = 26,      // [x * 4 + warp & 3] both halves' maxima (or sums) are there
  kNumBars = 34
};
constexpr uint32_t kUnitReaders = 19;   // MMA, K, V, sixteen softmax warps
constexpr int kOffTmem = 8 * kNumBars;  // TMEM base, abort flag
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffClc = 288;            // response (16 bytes, aligned)
constexpr int kOffUnits = 320;          // two descriptors
constexpr int kEmptySlots = 256;
constexpr int kOrdered = 64;            // prompts whose units are ordered as a whole

// What a unit is (in shared memory).
struct Unit {
  int live;       // 0: no more units
  int kvh, q0;    // kv head, first row of the prompt
  int rows, tile; // rows of the prompt, and which two Q tiles of them
  int end;        // rows [0, end) are seen
  int tiles;      // K/V tiles
};
static_assert(sizeof(Unit) <= 64 && kOffUnits + 2 * 64 <= 512 && kOffAbort + 4 <= kOffClc, "layout");

struct PromptArgs {
  const int32_t* qsl;
  int N, Hq, Hkv, grp;
  int row_tokens;             // query rows of a Q tile: 128 / grp
  int hkv_log2, per_log2;     // of Hkv and 2 * row_tokens where powers of two, else -1
  int total_q, max_query_len;
  int slots;                  // of the grid, per head
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

template <int D>
__global__ void __launch_bounds__(640, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map,
                 const __grid_constant__ PromptArgs a) {
  using C = PromptCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint8_t* ctl = smem + C::kOffBar;
  const uint32_t bars = sbase + C::kOffBar;
  auto BAR = [&](int k) { return bars + 8u * static_cast<uint32_t>(k); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + kOffAbort);
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
      tc::mbar_init(BAR(kPLo + b), 8);   // (warps)
      tc::mbar_init(BAR(kPHi + b), 8);
      tc::mbar_init(BAR(kODone + b), 1);
      tc::mbar_init(BAR(kUnitFull + b), 1);
      tc::mbar_init(BAR(kUnitEmpty + b), kUnitReaders);
    }
    tc::mbar_init(BAR(kClc), 1);
    tc::mbar_init(BAR(kFinal), 1);
    for (int k = 0; k < 8; ++k) tc::mbar_init(BAR(kPair + k), 2);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  // Which query row of the tile (past every prompt's where none) and head of the group a
  // TMEM lane is.
  if (threadIdx.x < C::kBM) {
    const int tok = static_cast<int>(threadIdx.x) / a.grp;
    reinterpret_cast<int2*>(smem + C::kOffRows)[threadIdx.x] =
        make_int2(tok < a.row_tokens ? tok : 1 << 30, static_cast<int>(threadIdx.x) - tok * a.grp);
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
    tc::reg_alloc<C::kRegSoftmax>();
    const int x = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
    // Registers are short while a tile's S is held, and what is spilled comes back from L2:
    // row() of the tile (= TMEM lane) is read anew where a unit begins and ends.
    auto row = []() -> int {
      uint32_t t;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
      return static_cast<int>(t & 127u);
    };
    auto row_is = [&](int t) {
      int2 v;
      asm volatile("ld.shared.v2.s32 {%0, %1}, [%2];"
                   : "=r"(v.x), "=r"(v.y)
                   : "r"(sbase + C::kOffRows + t * 8));
      return v;
    };
    // This half's columns of S (and P over them) and of O.
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + C::col_s(x) + 64 * half;
    const uint32_t to = ts + C::col_o(0) - C::col_s(0) - (64 - D / 2) * half;
    const int pair = kPair + x * 4 + (warp & 3);
    // This row and half in [tile & 1][x][half][128]; the other half's is 512 bytes apart.
    const uint32_t maxima = sbase + C::kOffMax + (x * 256 + half * 128 + (threadIdx.x & 127)) * 4;
    auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
      const bool w = __all_sync(0xffffffffu, tc::mbar_wait(b, parity));
      if (!w) fail();
      return w;
    };
    uint32_t g = 0, full = 0;   // tiles, units with tiles so far (exchanges: their sum)
    for (int u = 0;; ++u) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      if (!wait_warp(BAR(kUnitFull + (u & 1)), (u >> 1) & 1)) break;
      volatile Unit* un = unit_slot(u);
      if (!un->live) break;
      int seen = -64 * half;   // of a tile's columns of this half
      {
        const int tok = row_is(row()).x, q = (un->tile * 2 + x) * a.row_tokens;
        seen += tok < un->rows - q ? q + tok + 1 : 0;
      }
      // l: this half's sum of weights (for the LSE); lr: the same weights rounded to
      // bf16, as PV multiplies them (the output's divisor).
      float m_used = -CUDART_INF_F, l = 0.f, lr = 0.f;
      bool alive = true;
      for (int left = un->tiles; left > 0; --left, ++g) {
        if (!wait_warp(BAR(kSFull + x), g & 1)) {
          alive = false;
          break;
        }
        tc::tc_fence_after();
        uint32_t r[2][32];
        float m0, m1;
        tmem_ld32_max(ts, r[0], m0);
        tmem_ld32_max(ts + 32, r[1], m1);
        tc::tmem_wait_ld();
        if (__any_sync(0xffffffffu, seen < 64)) {
          m0 = m1 = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            r[0][c] = c < seen ? r[0][c] : 0xff800000u;   // -inf
            r[1][c] = 32 + c < seen ? r[1][c] : 0xff800000u;
            m0 = fmaxf(m0, __uint_as_float(r[0][c]));
            m1 = fmaxf(m1, __uint_as_float(r[1][c]));
          }
        }
        seen -= C::kBN;
        // weights(c): exp2(s * scale_log2 - m) in the place of s, of 32 columns.
        auto weights = [&](int c, float m) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1]), a.scale_log2, -m);
            r[c][e] = __float_as_uint(ex2(x0));
            r[c][e + 1] = __float_as_uint(ex2(x1));
          }
        };
        auto pack = [&](int c) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              pk[e] = pack_bf16(__uint_as_float(r[c][16 * q + 2 * e]),
                                __uint_as_float(r[c][16 * q + 2 * e + 1]));
            tmem_st8(ts + c * 16 + q * 8, pk);
          }
        };
        // The row's maximum over both halves.
        float mx = fmaxf(m0, m1) * a.scale_log2;
        const uint32_t mine = maxima + (g & 1) * 2048;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine), "f"(mx) : "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(BAR(pair));
        float mu = m_used == -CUDART_INF_F ? 0.f : m_used;
        if (!wait_warp(BAR(pair), (g + full) & 1)) {
          alive = false;
          break;
        }
        float others;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(others) : "r"(mine ^ 512u) : "memory");
        mx = fmaxf(mx, others);
        const bool need = mx > m_used + 8.f;
        float alpha = 1.f;
        if (__any_sync(0xffffffffu, need)) {
          if (need) {
            alpha = ex2(m_used - mx);
            mu = m_used = mx;
          }
          // S_x(j) has landed, hence PV_x(j-1) too: O_x may be rescaled now.
          if (left < un->tiles) {
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                uint32_t o[16];
                tmem_ld16(to + c * 32 + q * 16, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tc::tmem_st16(to + c * 32 + q * 16, o);
              }
            }
          }
        }
        weights(0, mu);
        // V rows behind the unit's last one may hold anything (0 * NaN is NaN):
        // cleared once V has landed, half a row per thread, before P is published.
        if (const int t = left > 1 ? 0 : row(); left == 1 && (un->tiles - 1) * C::kBN + t >= un->end) {
          if (!tc::mbar_wait(BAR(kVFull + (g & 1)), (g >> 1) & 1)) fail();
          const uint32_t vbase = sbase + C::kOffV + (g & 1) * C::kTileBytes;
#pragma unroll 1
          for (int c = half * (D / 16); c < (half + 1) * (D / 16); ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                             vbase + (c >> 3) * (C::kBN * 128) + sw128(t, c & 7)),
                         "r"(0u)
                         : "memory");
          tc::fence_proxy_async_smem();   // before this thread's P arrival
        }
        // P as bf16 pairs over this half's first 32 columns.
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          pack(c);
          if (c == 0) weights(1, mu);
          tc::tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(BAR((c == 0 ? kPLo : kPHi) + x));
        }
        // The sums, while the MMAs run.
        float l8[2] = {0.f, 0.f}, r8[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = __uint_as_float(r[c][e]), p1 = __uint_as_float(r[c][e + 1]);
            fadd2(l8[0], l8[1], p0, p1);
            add_bf16x2_f32(r8[0], r8[1], pack_bf16(p0, p1));
          }
        l = l * alpha + (l8[0] + l8[1]);
        lr = lr * alpha + (r8[0] + r8[1]);
      }
      const bool some = un->tiles > 0;
      if (alive && some) {
        // Both halves' sums.
        const uint32_t sums = sbase + C::kOffSum + (x * 256 + half * 128 + row()) * 8;
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sums), "f"(l), "f"(lr)
                     : "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(BAR(pair));
        alive = wait_warp(BAR(pair), (g + full) & 1);
        float ol, olr;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(ol), "=f"(olr)
                     : "r"(sums + 1024 - 2048 * half)
                     : "memory");
        l += ol;
        lr += olr;
        if (alive) alive = wait_warp(BAR(kODone + x), full & 1);
        ++full;
      }
      if (alive && some) {   // warp-uniform
        tc::tc_fence_after();
        const int2 is = row_is(row());
        const int q = (un->tile * 2 + x) * a.row_tokens;
        const bool valid = is.x < un->rows - q;
        const int64_t qrow = static_cast<int64_t>(un->q0 + q + is.x) * a.Hq + un->kvh * a.grp + is.y;
        // (A row with a visible token has a weight of 1.)
        const float inv = lr == 0.f ? 0.f : __fdividef(1.f, lr);
        // Two lanes store 64 bytes of a row, first of the even lane's, then of the odd one's:
        // they exchange half of what they have.  (Each its own row, 32 bytes in each of 32
        // lines for a store, kept the load and store unit busy: 16 prompts 211 us, so 202.)
        // 32-byte stores write whole sectors where `out` is 32-byte aligned.
        const bool a32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        const bool odd = lane & 1;
        auto mine = reinterpret_cast<unsigned long long>(a.out + qrow * D + half * (D / 2));
        if (!valid) mine = 0;
        auto other = __shfl_xor_sync(0xffffffffu, mine, 1);
        if (odd) {
          const auto m = mine;
          mine = other;
          other = m;
        }
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32], w[2][8];
          tc::tmem_ld32(to + c * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t lo = pack_bf16(__uint_as_float(o[2 * e]) * inv,
                                          __uint_as_float(o[2 * e + 1]) * inv);
            const uint32_t hi = pack_bf16(__uint_as_float(o[16 + 2 * e]) * inv,
                                          __uint_as_float(o[16 + 2 * e + 1]) * inv);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            w[0][e] = odd ? got : lo;
            w[1][e] = odd ? hi : got;
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint32_t* p = reinterpret_cast<uint32_t*>(v ? other : mine);
            if (p == nullptr) continue;
            p += c * 16 + odd * 8;
            if (a32) {
              st_global_v8(p, w[v]);
            } else {
              reinterpret_cast<uint4*>(p)[0] = make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]);
              reinterpret_cast<uint4*>(p)[1] = make_uint4(w[v][4], w[v][5], w[v][6], w[v][7]);
            }
          }
        }
        if (valid && half == 0 && a.lse != nullptr)
          a.lse[qrow] = l == 0.f ? -CUDART_INF_F : (m_used + __log2f(l)) * kLn2;
      }
      // The output's TMEM reads come before this warp's next P arrival, which the
      // next unit's first PV waits for.
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR(kUnitEmpty + (u & 1)));   // (it has been read)
      if (!alive) break;
    }
  } else {
    tc::reg_dealloc<C::kRegOther>();
    if (warp == 0) {
      // ------------------------------------------------------------ MMA issue
      if (elect_one()) {
        constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, C::kBN, 0, 0);
        constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, 0, 1);
        uint32_t g = 0, full = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t parity) { return tc::mbar_wait(BAR(bar), parity); };
        // Low words of the descriptors at the buffers' starts (offset 16 for the unused
        // leading dimension of Q and K, a column group for V).
        const uint32_t q_lo = (sbase >> 4) | (1u << 16);
        const uint32_t k_lo = ((sbase + C::kOffK) >> 4) | (1u << 16);
        const uint32_t v_lo = ((sbase + C::kOffV) >> 4) | ((C::kBN * 128 / 16) << 16);
        auto issue_s = [&](int x, uint32_t n) {
          const uint32_t ql = q_lo + x * (C::kQBytes >> 4);
          const uint32_t kl = k_lo + (n & 1) * (C::kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + C::col_s(x), ql + (((k >> 2) * (C::kBM * 128) + (k & 3) * 32) >> 4),
                   desc_hi(1024), kl + (((k >> 2) * (C::kBN * 128) + (k & 3) * 32) >> 4),
                   desc_hi(1024), idesc_s, k > 0);
          tc::mma_commit(BAR(kSFull + x));
        };
        // O_x (+)= P_x V over the 16-token steps of a part: 0, 1, 4, 5 or 2, 3, 6, 7
        // (each half's P lies over its own S columns).
        auto issue_pv = [&](int x, uint32_t n, auto part, bool fresh) {
          const uint32_t vl = v_lo + (n & 1) * (C::kTileBytes >> 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 2 * part + (e & 1) + 4 * (e >> 1);
            mma_ts(tmem + C::col_o(x), tmem + C::col_s(x) + (k >> 2) * 64 + (k & 3) * 8,
                   vl + k * (2048 >> 4), desc_hi(1024), idesc_o, !fresh || e > 0);
          }
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
            const bool more = j + 1 < ntiles;
            if (!wait(kVFull + (g & 1), (g >> 1) & 1)) { ok = false; break; }
            if (more && !wait(kKFull + ((g + 1) & 1), ((g + 1) >> 1) & 1)) { ok = false; break; }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!wait(kPLo + x, g & 1)) { ok = false; break; }
              tc::tc_fence_after();
              issue_pv(x, g, Step<0>(), j == 0);
              if (!wait(kPHi + x, g & 1)) { ok = false; break; }
              tc::tc_fence_after();
              issue_pv(x, g, Step<1>(), false);
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
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------ K, V
      if (lane == 0) {
        const bool is_v = warp == 3;
        const CUtensorMap* map = is_v ? &v_map : &k_map;
        const int full_bar = is_v ? kVFull : kKFull, empty_bar = is_v ? kVEmpty : kKEmpty;
        const uint32_t ring = sbase + (is_v ? C::kOffV : C::kOffK);
        uint32_t g = 0;
        bool ok = true;
        for (int u = 0; ok; ++u) {
          if (*abort_flag || !tc::mbar_wait(BAR(kUnitFull + (u & 1)), (u >> 1) & 1)) {
            ok = false;
            break;
          }
          volatile Unit* un = unit_slot(u);
          const int live = un->live, ntiles = un->tiles, q0 = un->q0, kvh = un->kvh;
          tc::mbar_arrive(BAR(kUnitEmpty + (u & 1)));
          if (!live) break;
          for (int j = 0; j < ntiles; ++j, ++g) {
            const uint32_t st = g & 1;
            if (*abort_flag ||
                (g >= 2 && !tc::mbar_wait(BAR(empty_bar + st), ((g >> 1) - 1) & 1))) {
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(BAR(full_bar + st), C::kTileBytes);
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tc::tma_load_3d(ring + st * C::kTileBytes + h * (C::kBN * 128), map, BAR(full_bar + st),
                              h * 64, kvh, q0 + j * C::kBN);
          }
        }
        if (!ok && !*abort_flag) fail();
        // No copy may still be landing when the CTA exits.
        for (uint32_t n = g >= 2 ? g - 2 : 0; n < g; ++n)
          if (!tc::mbar_wait(BAR(full_bar + (n & 1)), (n >> 1) & 1)) fail();
      }
    } else {
      // ------------------------------------------------------ units and queries
      // A slot of the grid is a unit of some prompt; the kv heads of a slot run side by
      // side (they read neighbouring parts of the same rows).
      const int per = 2 * a.row_tokens;
      auto rows_of = [&](int i, int& q0) {
        q0 = a.qsl[i];
        const int n = q0 >= 0 ? min(min(a.qsl[i + 1] - q0, a.max_query_len), a.total_q - q0) : 0;
        return max(0, n);
      };
      auto tiles_of = [&](int i) {
        int q0;
        return i < a.N ? div_bs(rows_of(i, q0) + per - 1, per, a.per_log2) : 0;
      };
      const bool ordered = a.N <= kOrdered;
      const int t0 = ordered ? tiles_of(lane) : 0, t1 = ordered ? tiles_of(lane + 32) : 0;
      const int levels = ordered ? __reduce_max_sync(0xffffffffu, max(t0, t1)) : 0;
      // Units of all prompts at places >= v of them.
      auto above = [&](int v) {
        return __reduce_add_sync(0xffffffffu, max(0, t0 - v) + max(0, t1 - v));
      };
      const uint32_t resp = bars + kOffClc;
      bool ok = true, asked = false;
      uint32_t answers = 0, full = 0, fetched = 0;   // fetched: Q tiles, 0 and 1 in turn
      int empty = 0;
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
      int slot = div_bs(blockIdx.x, a.Hkv, a.hkv_log2), head = blockIdx.x - slot * a.Hkv;
      ask();
      int u = 0;
      for (bool live = true; live;) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) {
          ok = false;
          break;
        }
        int request = -1, tile = 0;
        if (ordered) {
          // Units in the order of their places, the last first: slot s is at the highest
          // place v with above(v) > s, and there the (s - above(v + 1))-th prompt.
          if (slot < above(0)) {
            int lo = 0, hi = levels;   // above(lo) > slot >= above(hi)
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (above(mid) > slot) lo = mid; else hi = mid;
            }
            tile = lo;
            int k = slot - above(lo + 1);
            unsigned in = __ballot_sync(0xffffffffu, t0 > lo);
            const unsigned in1 = __ballot_sync(0xffffffffu, t1 > lo);
            int first = 0;
            if (k >= __popc(in)) {
              k -= __popc(in);
              in = in1;
              first = 32;
            }
            request = first + static_cast<int>(__fns(in, 0, k + 1));
          }
        } else {
          // Slot s belongs to the last prompt i with qsl[i] / per + i <= s: prompt i owns
          // at least ceil(rows / per) slots from there on.  Counted from the end, so that
          // a prompt's later units come first.
          const int s = a.slots - 1 - slot;
          int lo = 0, hi = a.N;
          for (;;) {
            const int step = (hi - lo + 31) / 32, i = lo + lane * step;
            const int q = i < hi ? a.qsl[i] : 0;
            const unsigned below =
                __ballot_sync(0xffffffffu, i < hi && div_bs(q, per, a.per_log2) + i <= s);
            const int k = max(31 - __clz(below), 0);
            lo += k * step;
            hi = min(lo + step, hi);
            if (step == 1) break;
          }
          tile = s - (div_bs(a.qsl[lo], per, a.per_log2) + lo);
          request = tile >= 0 ? lo : -1;
        }
        int q0 = 0;
        const int rows = request >= 0 ? rows_of(request, q0) : 0;
        const int qi = tile * per;
        const bool real = request >= 0 && qi < rows;
        // A long run of empty slots is broken by units without rows, so that the other
        // warps' waits for a unit stay short.
        empty = real ? 0 : empty + 1;
        if (real || empty == kEmptySlots) {
          empty = 0;
          const int end = real ? min(qi + per, rows) : 0;
          const int tiles = (end + C::kBN - 1) / C::kBN;
          if (u >= 2 &&
              !__all_sync(0xffffffffu, wait(kUnitEmpty + (u & 1), ((u >> 1) - 1) & 1))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            volatile Unit* un = unit_slot(u);
            un->live = 1;
            un->kvh = head;
            un->q0 = q0;
            un->rows = real ? rows : 0;
            un->tile = tile;
            un->end = end;
            un->tiles = tiles;
            tc::mbar_arrive(BAR(kUnitFull + (u & 1)));
          }
          __syncwarp();
          ++u;
          if (tiles > 0) {
            // Rows past the prompt or the batch are fetched too (or zeros): they are masked.
            for (int x = 0; x < 2 && ok; ++x) {
              if (full > 0 && !__all_sync(0xffffffffu, wait(kQEmpty + x, (full - 1) & 1))) {
                ok = false;
                break;
              }
              if (lane == 0) {
                tc::mbar_arrive_expect_tx(
                    BAR(kQFull + x), static_cast<uint32_t>(a.row_tokens * a.grp) * (D * 2));
                for (int h = 0; h < C::kHalves; ++h)
                  tc::tma_load_3d(sbase + x * C::kQBytes + h * (C::kBM * 128), &q_map,
                                  BAR(kQFull + x), h * 64, head * a.grp,
                                  min(q0 + qi + x * a.row_tokens, a.total_q));
              }
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
        for (int x = 0; x < 2; ++x) {
          const uint32_t n = (fetched + 1 - x) >> 1;
          if (n > 0) tc::mbar_wait(BAR(kQFull + x), (n - 1) & 1);
        }
      }
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

// Rows [T][H][d] with `stride` elements from token to token: 64 columns x `heads` heads
// x `rows` tokens.
bool make_rows_map(CUtensorMap* map, const void* p, int T, int H, int d, int64_t stride, int heads,
                   int rows) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_t(const PromptLaunch& n, cudaStream_t stream) {
  using C = PromptCfg<D>;
  PromptArgs a{};
  a.qsl = n.qsl;
  a.N = n.N;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.grp = n.Hq / n.Hkv;
  a.row_tokens = C::kBM / a.grp;
  a.hkv_log2 = block_size_log2(n.Hkv);
  a.per_log2 = block_size_log2(2 * a.row_tokens);
  a.total_q = n.total_q;
  a.max_query_len = n.max_query_len;
  a.scale_log2 = n.scale * kLog2e;
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  CUtensorMap q_map, k_map, v_map;
  if (!make_rows_map(&q_map, n.q, n.total_q, n.Hq, D, n.q_stride, a.grp, a.row_tokens) ||
      !make_rows_map(&k_map, n.key, n.total_q, n.Hkv, D, n.key_stride, 1, C::kBN) ||
      !make_rows_map(&v_map, n.value, n.total_q, n.Hkv, D, n.value_stride, 1, C::kBN))
    return cudaErrorInvalidValue;
  auto kern = prompt_tc_kernel<D>;
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  // The register hand-over between warpgroups waits for registers that the launch must
  // actually hold; refuse to launch a build that does not.
  static const bool regs_ok = [&] {
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return false;
    const long long have = static_cast<long long>(fa.numRegs) * C::kThreads;
    const long long need = 512LL * C::kRegSoftmax + 128LL * C::kRegOther;
    return fa.numRegs >= static_cast<int>(C::kRegOther) &&
           fa.numRegs <= static_cast<int>(C::kRegSoftmax) && have >= need;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  const long long slots = n.total_q / (2 * a.row_tokens) + static_cast<long long>(n.N);
  if (slots * n.Hkv > INT_MAX) return cudaErrorInvalidValue;
  a.slots = static_cast<int>(slots);
  return launch_pdl(kern, dim3(static_cast<unsigned>(slots * n.Hkv)), dim3(C::kThreads),
                    C::kSmemBytes, stream, q_map, k_map, v_map, a);
}

}  // namespace

cudaError_t launch_prompt(const PromptLaunch& n, cudaStream_t stream) {
  return n.d == 64 ? launch_t<64>(n, stream) : launch_t<128>(n, stream);
}

}  // namespace pa
