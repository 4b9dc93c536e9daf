// Decode attention over a 4-bit pool (layout: fp4.cuh): o = softmax(scale q K^T) V
// for one query per request, with K, V = code * scale * k_scale (v_scale).
//
// The work is one line of 16-token pieces: request by request, kv head by kv head,
// token by token.  It is cut into as many equal parts as CTAs are resident, whatever
// the lengths, and a part into eight for the CTA's warps: each finds its place from the
// lengths' sum (a scan) and walks over the (request, kv head) units in it by itself.  A
// unit that lies with one warp gives its output at once.  Of one that is cut the warps
// keep states (o, maximum, sum), which the CTA merges at its end, and what is cut
// between CTAs a second kernel: two states per CTA at most, however long the context.
// (One CTA per unit and split, dealt by the hardware, left SMs idle for a quarter of
// the time on 64 requests of U[128, 4096] tokens, with a quarter of the instructions in
// CTAs' ends; a CTA's warps side by side in one unit waited for each other at each
// unit's end, longest where requests are short: 65 us against 52.)
//
// A warp fetches its own slices of 32 tokens: two pieces (keys, values and scales of 16
// tokens are one run of 18 d bytes: one bulk copy) into a ring of its own.  It takes
// them as two M = 16 tiles of mma.m16n8k16 with the group's query heads as N (8 per
// n-tile): S^T = K Q^T, one online softmax step over the 32 tokens, O^T += V^T P^T.
// Codes are widened to f16 and multiplied by their scales on the way into operand
// registers (exact); q and the weights are f16.
//
// Bound by issue slots beside HBM: 2304 bytes for 16 tokens (d = 128) pass in 100
// cycles of an SM, in which it issues 400 warp instructions, 200 of them on the ALU,
// and a piece needs 64 conversions (ALU), 64 scalings and 16 MMAs before anything else.
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "pa_launch.h"
#include "tc_tiles.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPieces = 2;                   // 16-token pieces of a warp's slice
constexpr int kSlice = 16 * kPieces;         // tokens
// What a unit's start and end cost a warp, in pieces: it counts on the line in front of
// the unit's tokens.  (128 requests of U[1, 8191]
// tokens, 64-wide heads: 100 us with 0, 94 with 2, 90 with 4 to 8.)
constexpr int kExtra = 6;

struct Fp4Args {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int N, max_blocks, Hq, Hkv, grp, bs, bs_log2, num_blocks;
  int whole;          // units are not cut between CTAs
  int positions;      // of a table row, at most INT_MAX - 1023
  float scale_log2;   // scale * k_scale * log2(e)
  float out_scale;    // v_scale
  float4* held;       // [CTA][warp] states of units that began with an earlier warp
  float* parts;       // [CTA][2][grp][d + 2] states of units that are cut between CTAs
  int4* cut;          // [CTA]: (first CTA, request, kv head) of the unit whose end it holds
  int2* spans;        // [N, Hkv] first and last CTA of a unit, or null
  float* row_lse;     // [N, Hq] of units that are not cut, with spans
  float* logits;      // [N, Hkv, logit_tokens, grp] (log2 units), or null
  int logit_tokens;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

template <int D, int NT>
struct Fp4Cfg {
  static constexpr int kPairBytes = 2 * fp4::tile_bytes(D);
  static constexpr int kSlotBytes = kPieces * kPairBytes;
  static constexpr int kCtas = NT == 1 ? 2 : 1;                    // per SM
  static constexpr int kSlots = (D == 128 ? 3 : 6) * (2 / kCtas);  // of a warp's ring
  static constexpr int kRingBytes = kWarps * kSlots * kSlotBytes;
  // A state: for each n-tile o, then maxima and sums, 16 bytes a lane at a time.
  static constexpr int kStateVecs = NT * (D / 16 + 1) * 32;
  static_assert(kStateVecs * 16 <= kSlots * kSlotBytes, "a state fits a warp's ring");
  static constexpr int kOffBar = kRingBytes;
  static constexpr int kOffPlaces = kOffBar + 8 * kWarps * kSlots;
  static constexpr int kSmemBytes = kOffPlaces + 512;
};

// Where in the line something is: a request and the pieces before it in that request's
// units.
struct Place {
  long long inside;
  int i, pad;
};
// What a warp has kept for the CTA's merge.
struct Kept {
  long long begin;     // of the unit, in the line
  int i, h;
  int where;           // 0: nothing, 1: in memory, 2: in the warp's ring
  int ends;
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

// x / n; 64-bit divisions take a hundred instructions.
__device__ __forceinline__ long long quotient(long long x, long long n) {
  return (x | n) <= INT_MAX ? static_cast<int>(x) / static_cast<int>(n) : x / n;
}

// Where a warp (or its fetches, ahead of it) stands in its part of the line.
struct Walk {
  int i, h;            // unit
  int seq, after;      // tokens of request i and of request i + 1
  int tok, end;        // its tokens in this part
  int left;            // of the part behind the unit
};

__device__ __forceinline__ int length_of(const Fp4Args& a, int i) {
  // What lies past the table's columns has no block and is not walked over.
  return i < a.N ? min(max(0, a.seq_lens[i]), a.positions) : 0;
}
// Enters the unit at `at` on its stretch of the line (kExtra, then its pieces); false
// where the part ends before its tokens.
__device__ __forceinline__ bool walk_enter(Walk& w, int at) {
  const int skip = max(0, kExtra - at), from = max(0, at - kExtra);
  const int pieces = ((w.seq + 15) >> 4) - from, mine = w.left - skip;
  w.tok = 16 * from;
  w.end = mine < pieces ? 16 * (from + mine) : w.seq;
  w.left -= skip + pieces;
  return mine > 0;
}
// On to the next unit with tokens; false at the part's end.
__device__ __forceinline__ bool walk_next(const Fp4Args& a, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.h == a.Hkv) {
    w.h = 0;
    do {
      if (++w.i >= a.N) return false;   // (lengths that changed under way)
      w.seq = w.after;
      w.after = length_of(a, w.i + 1);
    } while (w.seq == 0);
  }
  return walk_enter(w, 0);
}

// A warp's running state; a lane holds the heads nt * 8 + 2 tid4 + {0, 1}, and of each
// the D / 8 neighbouring dims from gid * (D / 8) on.
template <int D, int NT>
struct Fp4State {
  float m[NT][2], l[NT][2], o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int md = 0; md < D / 16; ++md)
        o[nt][md][0] = o[nt][md][1] = o[nt][md][2] = o[nt][md][3] = 0.f;
    }
  }
  // 16 bytes a lane at a time.
  __device__ __forceinline__ void store(float4* p, int lane) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int md = 0; md < D / 16; ++md)
        p[(nt * (D / 16 + 1) + md) * 32 + lane] =
            make_float4(o[nt][md][0], o[nt][md][1], o[nt][md][2], o[nt][md][3]);
      p[(nt * (D / 16 + 1) + D / 16) * 32 + lane] =
          make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
    }
  }
  // The finished rows of unit (i, h).
  __device__ __forceinline__ void output(const Fp4Args& a, int i, int h, int lane) const {
    const int gid = lane >> 2, tid4 = lane & 3;
    const int64_t row0 = static_cast<int64_t>(i) * a.Hq + h * a.grp;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * tid4 + j;
        if (r >= a.grp) continue;
        const float f = l[nt][j] == 0.f ? 0.f : a.out_scale / l[nt][j];
        __nv_bfloat16* dst = a.out + (row0 + r) * D + gid * (D / 8);
        if ((reinterpret_cast<uintptr_t>(a.out) & 15u) == 0) {
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16(o[nt][4 * k + e][j] * f, o[nt][4 * k + e][2 + j] * f);
            reinterpret_cast<uint4*>(dst)[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int md = 0; md < D / 16; ++md) {
            dst[2 * md] = __float2bfloat16_rn(o[nt][md][j] * f);
            dst[2 * md + 1] = __float2bfloat16_rn(o[nt][md][2 + j] * f);
          }
        }
        if (gid == 0) {
          const float x = l[nt][j] == 0.f ? -CUDART_INF_F : (m[nt][j] + log2f(l[nt][j])) * kLn2;
          if (a.lse != nullptr) a.lse[row0 + r] = x;
          if (a.spans != nullptr) a.row_lse[row0 + r] = x;
        }
      }
    if (a.spans != nullptr && lane == 0)
      a.spans[static_cast<int64_t>(i) * a.Hkv + h] = make_int2(blockIdx.x, blockIdx.x);
  }
};

template <int D, int NT, bool LOGITS>
__global__ void __launch_bounds__(kThreads, Fp4Cfg<D, NT>::kCtas) decode_fp4_kernel(
    const __grid_constant__ Fp4Args a) {
  using C = Fp4Cfg<D, NT>;
  constexpr int kK = D / 16;          // k-steps of K Q^T = d-tiles of V^T P^T
  constexpr int kWk = D / 32;         // words of a key row in a lane: D / 4 codes
  constexpr int kWv = D / 64;         // words of a value row in a lane: D / 8 codes
  constexpr float kRescale = 8.f;     // log2 units
  extern __shared__ __align__(128) uint8_t smem[];
  const int cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;
  const int grp = a.grp;
  const uint32_t ring = smem_u32(smem) + warp * C::kSlots * C::kSlotBytes;
  const uint32_t bars = smem_u32(smem) + C::kOffBar + warp * C::kSlots * 8;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < C::kSlots; ++k) tc::mbar_init(bars + 8 * k, 1);
    tc::fence_barrier_init();
  }
  __syncwarp();   // each warp uses its own barriers only
  pdl_wait();
  pdl_trigger();

  // ------------------------------------------------------------ the part
  // (Code that runs once is slow, it is fetched as it goes: loops are kept as loops.)
  // Requests are dealt over the threads that scan, neighbouring ones to each: those of a
  // warp by itself where they are few, else those of the CTA.
  const bool few = a.N <= 256;
  const int scanner = few ? lane : threadIdx.x, scanners = few ? 32 : kThreads;
  const int chunk = (a.N + scanners - 1) / scanners;
  const int r0 = min(a.N, scanner * chunk), r1 = min(a.N, r0 + chunk);
  auto weight = [&](int seq) { return seq > 0 ? kExtra + ((seq + 15) >> 4) : 0; };
  long long mine = 0;
  for (int i = r0; i < r1; ++i) mine += weight(length_of(a, i));
  mine *= a.Hkv;
  long long before = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  long long total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  Place* found = reinterpret_cast<Place*>(smem + C::kOffPlaces);   // (not few: for one warp at a time)
  if (!few) {
    long long* scan = reinterpret_cast<long long*>(smem + C::kOffPlaces);
    if (lane == 31) scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
  }
  // The place of position g < total.  Few: g is the warp's own; else the CTA's, one
  // after another.
  auto locate = [&](long long g) {
    const bool here = g >= before && g < before + mine;
    int i = r0;
    long long in = g - before;
    if (few) {
      const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      i = __shfl_sync(0xffffffffu, i, src);
      in = __shfl_sync(0xffffffffu, in, src);
    }
    if (few || here)
      for (; i + 1 < a.N; ++i) {
        const long long n = static_cast<long long>(weight(length_of(a, i))) * a.Hkv;
        if (in < n) break;
        in -= n;
      }
    Place p{in, i, 0};
    if (!few) {
      __syncthreads();   // the last one has been read
      if (here) *found = p;
      __syncthreads();
      p = *found;
    }
    return p;
  };
  // Parts of equal length, in whole slices.
  const long long share = (quotient(total + gridDim.x - 1, gridDim.x) + kPieces - 1) / kPieces * kPieces;
  long long g0 = min(total, cta * share), g1 = min(total, g0 + share);
  if (a.whole) {
    // The units that begin in the part.
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      long long& g = k == 0 ? g0 : g1;
      if (g < total) {
        const Place p = locate(g);
        const int n = weight(length_of(a, p.i));
        const int in = static_cast<int>(p.inside - quotient(p.inside, n) * n);
        g += in > 0 ? n - in : 0;
      }
    }
  }
  const long long per = ((g1 - g0 + kWarps - 1) / kWarps + kPieces - 1) / kPieces * kPieces;
  const long long w0 = g0 + warp * per, w1 = min(g1, w0 + per);
  bool any = w0 < w1;
  Place place{};
  if (few) {
    if (any) place = locate(w0);
  } else {
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w)
      if (g0 + w * per < g1) {   // CTA-uniform
        const Place p = locate(g0 + w * per);
        if (w == warp) place = p;
      }
    __syncthreads();   // the last place has been read
  }
  Kept* kept = reinterpret_cast<Kept*>(smem + C::kOffPlaces);   // [kWarps][unit began before, begins]
  if (lane < 2) kept[2 * warp + lane].where = 0;
  __syncwarp();
  if (cta == 0 && warp == 0) {
    bool past = false;
    for (int i = lane; i < a.N; i += 32) past |= a.seq_lens[i] > a.positions;
    if (past) record_error(a.err, PA_DEVERR_BLOCK_ID);
  }
  // Requests without tokens.
  for (int i = cta; i < a.N; i += gridDim.x)
    if (length_of(a, i) == 0) {
      for (int k = threadIdx.x; k < a.Hq * D; k += kThreads)
        a.out[static_cast<int64_t>(i) * a.Hq * D + k] = __float2bfloat16_rn(0.f);
      if (a.lse != nullptr)
        for (int k = threadIdx.x; k < a.Hq; k += kThreads)
          a.lse[static_cast<int64_t>(i) * a.Hq + k] = -CUDART_INF_F;
    }
  if (!a.whole && threadIdx.x == 0) a.cut[cta] = make_int4(-1, 0, 0, 0);
  Walk at{};
  long long pos = 0;   // of the unit's first token in the line
  if (any) {
    at.i = place.i;
    at.seq = length_of(a, at.i);
    at.after = length_of(a, at.i + 1);
    at.left = static_cast<int>(min(w1 - w0, static_cast<long long>(INT_MAX)));
    const int n = weight(at.seq);
    at.h = static_cast<int>(quotient(place.inside, n));
    const int in = static_cast<int>(place.inside - static_cast<long long>(at.h) * n);
    any = walk_enter(at, in);
    pos = w0 - in + kExtra;
  }
  Walk ahead = at;

  // ------------------------------------------------------------ fetches
  // Addresses are made for 32 pieces of a unit at a time, a lane's each: the block ids
  // are asked for with the last slice before, and turned into addresses with the next.
  const int64_t head_bytes = static_cast<int64_t>(a.bs >> 4) * C::kPairBytes;
  const int64_t block_bytes = head_bytes * a.Hkv;
  bool more = any;
  int tok = ahead.tok;     // of the next slice to be fetched
  int blk = -1, next = 0;  // the lane's block id; pieces of the 32 that are used up
  bool fresh = true;       // ... and whether it has been turned into an address
  uint32_t valid = 0;      // pieces of the 32 that are there
  const uint8_t* src = nullptr;
  auto lookup = [&]() {
    const int t = tok + 16 * lane;
    // (A plain load: the table may be the previous kernel's output.)
    blk = more && t < ahead.end ? a.block_table[static_cast<int64_t>(ahead.i) * a.max_blocks +
                                                div_bs(t, a.bs, a.bs_log2)]
                                : -1;
    fresh = true;
    next = 0;
  };
  lookup();
  int fill = 0;            // the slot that it goes to
  uint32_t loaded = 0;     // kPieces bits per slot: pieces that are there
  bool ok = true;          // (a warp that gave up fetches no more)
  int flying = 0;          // slices on their way
  auto fetch = [&]() {
    if (!more || !ok) return;
    if (fresh) {
      const bool good = blk >= 0 && blk < a.num_blocks;
      if (!good && tok + 16 * lane < ahead.end) record_error(a.err, PA_DEVERR_BLOCK_ID);
      valid = __ballot_sync(0xffffffffu, good);
      src = a.cache + ahead.h * head_bytes + (good ? blk : 0) * block_bytes +
            (mod_bs(tok + 16 * lane, a.bs, a.bs_log2) >> 4) * C::kPairBytes;
      fresh = false;
    }
    const uint32_t there = (valid >> next) & 3u;
    const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), next + lane);
    loaded = (loaded & ~(3u << (kPieces * fill))) | (there << (kPieces * fill));
    const uint32_t bar = bars + 8 * fill;
    if (lane == 0) tc::mbar_arrive_expect_tx(bar, __popc(there) * C::kPairBytes);
    __syncwarp();
    if ((there >> lane) & 1u)
      bulk_load(ring + fill * C::kSlotBytes + lane * C::kPairBytes,
                reinterpret_cast<const void*>(from), C::kPairBytes, bar);
    if (++fill == C::kSlots) fill = 0;
    ++flying;
    tok += kSlice;
    next += kPieces;
    if (tok >= ahead.end) {
      more = walk_next(a, ahead);
      tok = 0;             // (a part's later units are entered at their start)
      lookup();
    } else if (next == 32) {
      lookup();
    }
  };
#pragma unroll 1
  for (int k = 0; k < C::kSlots; ++k) fetch();

  // Source lanes of the P^T operand (tokens 2 tid4 and 2 tid4 + 1 of head gid).
  const int src_a = 8 * tid4 + (gid >> 1), src_b = src_a + 4;
  const uint32_t sel = (gid & 1) ? 0x7632u : 0x5410u;
  int slot = 0, parity = 0;   // of the slice worked on
  Fp4State<D, NT> st;
  // The unit's queries, as the B operand.
  uint32_t qf[NT][kK][2];
  auto queries = [&]() {
    const __nv_bfloat16* qb =
        a.q + (static_cast<int64_t>(at.i) * a.Hq + at.h * grp) * D + tid4 * (D / 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gid;
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        qf[nt][kk][0] = qf[nt][kk][1] = 0u;
        if (h < grp) {
          qf[nt][kk][0] = q_pair(qb + h * D + kk * 4);
          qf[nt][kk][1] = q_pair(qb + h * D + kk * 4 + 2);
        }
      }
    }
  };
  for (bool live = any; live;) {
    // ---------------------------------------------------------- one unit
    queries();
    st.clear();
    for (int tb = at.tok; tb < at.end; tb += kSlice) {
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(bars + 8 * slot, parity));
      if (!ok) continue;
      const uint32_t here = loaded >> (kPieces * slot);
      // Visible tokens of each piece.
      int lim[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        lim[p] = (here >> p) & 1u ? min(16, at.end - (tb + 16 * p)) : 0;
      const uint32_t pair = ring + slot * C::kSlotBytes;
      const bool whole = lim[0] == 16 && lim[1] == 16;
      // All loads of keys first: what follows waits for them once.
      uint32_t kw[kPieces][2][kWk], ksc[kPieces][2];
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint32_t kb = pair + p * C::kPairBytes, ks = kb + 8 * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = gid + 8 * h;
          ksc[p][h] = D == 128 ? lds_u16(ks + row * 8 + tid4 * 2) : lds_u8(ks + row * 4 + tid4);
          lds_words(kb + row * (D / 2) + tid4 * (D / 8), kw[p][h]);
        }
      }
      // S^T = K Q^T: rows = tokens gid, gid + 8; columns = heads.  Pieces and even and
      // odd k-steps in turn: four chains of MMAs.
      uint32_t ks[kPieces][2][2];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t c = fp4::widen_scales(ksc[p][h]);
          ks[p][h][0] = fp4::both_low(c), ks[p][h][1] = fp4::both_high(c);
        }
      float s2[kPieces][NT][2][4];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            s2[p][nt][h][0] = s2[p][nt][h][1] = s2[p][nt][h][2] = s2[p][nt][h][3] = 0.f;
#pragma unroll
      for (int w = 0; w < kWk; ++w)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          uint32_t f0[4], f1[4];
          fp4::widen8(kw[p][0][w], f0);
          fp4::widen8(kw[p][1][w], f1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t am[4] = {
                fp4::mul2(f0[2 * h], ks[p][0][w / 2]), fp4::mul2(f1[2 * h], ks[p][1][w / 2]),
                fp4::mul2(f0[2 * h + 1], ks[p][0][w / 2]), fp4::mul2(f1[2 * h + 1], ks[p][1][w / 2])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(s2[p][nt][h], am, qf[nt][2 * w + h][0], qf[nt][2 * w + h][1]);
          }
        }
      float x[kPieces][NT][4];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[p][nt][e] = (s2[p][nt][0][e] + s2[p][nt][1][e]) * a.scale_log2;
      // ... and of values, under the softmax.
      uint32_t v[kPieces][4][kWv], vsc[kPieces][4];
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint32_t vb = pair + p * C::kPairBytes + fp4::tile_bytes(D), vs = vb + 8 * D;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 2 * tid4 + (r & 1) + 8 * (r >> 1);
          vsc[p][r] = lds_u8(vs + row * (D / 16) + (D == 128 ? gid : gid >> 1));
          lds_words(vb + row * (D / 2) + gid * (D / 16), v[p][r]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gid + 8 * (e >> 1) >= lim[p]) x[p][nt][e] = -CUDART_INF_F;
      }
      if constexpr (LOGITS) {
        // (Of every token, also where a block is missing.)
        const int64_t unit = static_cast<int64_t>(at.i) * a.Hkv + at.h;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int tok = tb + 16 * p + gid;
          float* dst = a.logits + (unit * a.logit_tokens + tok) * grp;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = nt * 8 + 2 * tid4 + (e & 1);
              if (h < grp && tok + 8 * (e >> 1) < min(at.end, a.logit_tokens))
                dst[8 * (e >> 1) * grp + h] = x[p][nt][e];
            }
        }
      }
      // Online softmax in the log2 domain; the reference maximum moves only when the
      // 32 tokens' exceeds it by more than kRescale, so that weights stay < 2^8.
      uint32_t pb[kPieces][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[kPieces][4], mx[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y = fmaxf(fmaxf(x[0][nt][j], x[0][nt][2 + j]), fmaxf(x[1][nt][j], x[1][nt][2 + j]));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          mx[j] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
        }
        if (__any_sync(0xffffffffu, mx[0] > st.m[nt][0] + kRescale || mx[1] > st.m[nt][1] + kRescale)) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool up = mx[j] > st.m[nt][j] + kRescale;
            const float alpha = up ? ex2(st.m[nt][j] - mx[j]) : 1.f;   // 0 when the old one is -inf
            if (up) st.m[nt][j] = mx[j];
            st.l[nt][j] *= alpha;
#pragma unroll
            for (int md = 0; md < kK; ++md) {
              st.o[nt][md][j] *= alpha;
              st.o[nt][md][2 + j] *= alpha;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mu = st.m[nt][j] == -CUDART_INF_F ? 0.f : st.m[nt][j];
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
            pr[p][j] = ex2(x[p][nt][j] - mu);
            pr[p][2 + j] = ex2(x[p][nt][2 + j] - mu);
            st.l[nt][j] += pr[p][j] + pr[p][2 + j];
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
      // O^T += V^T P^T: a lane's codes are d / 8 neighbouring ones of the value rows 2
      // tid4, + 1, + 8, + 9; two tokens' codes are interleaved by halves of bytes.
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        if (!whole) {
          // The weight of a token that is not there is 0, its codes are finite whatever
          // the bytes, but its scale need not be.
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (2 * tid4 + (r & 1) + 8 * (r >> 1) >= lim[p]) vsc[p][r] = 0u;
        }
        const uint32_t sab = fp4::widen_scales(vsc[p][0] | (vsc[p][1] << 8));
        const uint32_t scd = fp4::widen_scales(vsc[p][2] | (vsc[p][3] << 8));
#pragma unroll
        for (int w = 0; w < kWv; ++w) {
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          uint32_t ab[2][4], cd[2][4];   // [even, odd element][word byte]
          fp4::widen8((v[p][0][w] & kLow) | ((v[p][1][w] << 4) & ~kLow), ab[0]);
          fp4::widen8(((v[p][0][w] >> 4) & kLow) | (v[p][1][w] & ~kLow), ab[1]);
          fp4::widen8((v[p][2][w] & kLow) | ((v[p][3][w] << 4) & ~kLow), cd[0]);
          fp4::widen8(((v[p][2][w] >> 4) & kLow) | (v[p][3][w] & ~kLow), cd[1]);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t am[4] = {fp4::mul2(ab[0][b], sab), fp4::mul2(ab[1][b], sab),
                                    fp4::mul2(cd[0][b], scd), fp4::mul2(cd[1][b], scd)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(st.o[nt][4 * w + b], am, pb[p][nt][0], pb[p][nt][1]);
          }
        }
      }
      __syncwarp();   // every lane has read the slot
      --flying;
      fetch();
      if (++slot == C::kSlots) slot = 0, parity ^= 1;
    }

    // ---------------------------------------------------------- its end
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1)
          st.l[nt][j] += __shfl_xor_sync(0xffffffffu, st.l[nt][j], k);
    const bool starts = at.tok == 0, ends = at.end == at.seq;
    const Walk was = at;
    live = walk_next(a, at);
    if (starts && ends) {
      st.output(a, was.i, was.h, lane);
    } else {
      // Kept until all warps are done: the last one in the ring, which is free by then.
      if (live)
        st.store(a.held + static_cast<int64_t>(cta * kWarps + warp) * C::kStateVecs, lane);
      else if (ok)
        st.store(reinterpret_cast<float4*>(smem + warp * C::kSlots * C::kSlotBytes), lane);
      if (lane == 0)
        kept[2 * warp + starts] = Kept{pos, was.i, was.h, live ? 1 : 2, ends};
    }
    pos += kExtra + ((was.seq + 15) >> 4);
  }
  if (!ok && lane == 0) {
    // Given up: the outputs are invalid.  No copy may still be landing when the ring is
    // read as a state or the CTA exits: what is on its way gets one more bounded wait each.
    record_error(a.err, PA_DEVERR_TIMEOUT);
    for (int k = 0; k < flying; ++k) {
      tc::mbar_wait(bars + 8 * slot, parity);
      if (++slot == C::kSlots) slot = 0, parity ^= 1;
    }
  }
  __syncthreads();
  // ------------------------------------------------------------ units cut between warps
  // Run 0: the unit that began in an earlier CTA; run k: the one that begins with warp
  // k - 1 and goes on.  A run is the state that begins it and the first states of the
  // warps behind, up to one that ends.
  auto state_of = [&](int w, int where) {
    return where == 1 ? a.held + static_cast<int64_t>(cta * kWarps + w) * C::kStateVecs
                      : reinterpret_cast<const float4*>(smem + w * C::kSlots * C::kSlotBytes);
  };
  // A warp takes a d-tile of each run.
#pragma unroll 1
  for (int run = 0; run <= kWarps; ++run) {
    const int from = run == 0 ? 0 : run - 1;
    const Kept first = kept[2 * from + (run > 0)];
    if (first.where == 0 || warp >= kK) continue;   // warp-uniform
    const bool starts = run > 0;
    bool ends = false;
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      float M[2] = {-CUDART_INF_F, -CUDART_INF_F}, L[2] = {0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
      ends = false;
#pragma unroll 1
      for (int w = from; w < kWarps && !ends; ++w) {
        const Kept* k = &kept[2 * w + (w == from && starts)];
        const int where = k->where;
        if (where == 0) break;
        ends = k->ends;
        const float4* p = state_of(w, where) + nt * (kK + 1) * 32 + lane;
        const float4 ml = p[kK * 32], o = p[warp * 32];
        const float m[2] = {ml.x, ml.y}, l[2] = {ml.z, ml.w}, v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float top = fmaxf(M[j], m[j]);
          // (Equal, also where both are -inf: 1.)
          const float f = M[j] == top ? 1.f : ex2(M[j] - top), g = m[j] == top ? 1.f : ex2(m[j] - top);
          M[j] = top;
          L[j] = f * L[j] + g * l[j];
          y[j] = f * y[j] + g * v[j];
          y[2 + j] = f * y[2 + j] + g * v[2 + j];
        }
      }
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * tid4 + j, dim = gid * (D / 8) + 2 * warp;
        const float l = j ? L[1] : L[0], m = j ? M[1] : M[0];
        const float y0 = j ? y[1] : y[0], y1 = j ? y[3] : y[2];
        if (r >= grp) continue;
        if (starts && ends) {
          const int64_t row = static_cast<int64_t>(first.i) * a.Hq + first.h * grp + r;
          const float f = l == 0.f ? 0.f : a.out_scale / l;
          a.out[row * D + dim] = __float2bfloat16_rn(y0 * f);
          a.out[row * D + dim + 1] = __float2bfloat16_rn(y1 * f);
          if (gid == 0 && warp == 0) {
            const float x = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
            if (a.lse != nullptr) a.lse[row] = x;
            if (a.spans != nullptr) a.row_lse[row] = x;
          }
        } else {
          float* dst = a.parts + ((static_cast<int64_t>(cta) * 2 + starts) * grp + r) * (D + 2);
          *reinterpret_cast<float2*>(dst + dim) = make_float2(y0, y1);
          if (gid == 0 && warp == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(m, l);
        }
      }
    }
    if (warp != 0 || lane != 0) continue;
    if (!starts && ends)
      a.cut[cta] = make_int4(static_cast<int>(quotient(first.begin, share)), first.i, first.h, 0);
    if (starts && a.spans != nullptr)
      a.spans[static_cast<int64_t>(first.i) * a.Hkv + first.h] = make_int2(
          cta, ends ? cta
                    : static_cast<int>(quotient(first.begin + ((length_of(a, first.i) + 15) >> 4) - 1,
                                             share)));
  }
}

// The states of a cut unit, one CTA for each CTA that holds a unit's end and each head:
// the first CTA's second state, then the following CTAs' first states up to this one's.
template <int D, int kAhead>
__device__ __forceinline__ void merge_cut(const Fp4Args& a, const int4& u, int c1, int r) {
  static_assert(kAhead <= D, "a thread for each state");
  __shared__ float factor[D];
  __shared__ float red[2][D / 32];
  const int e = threadIdx.x, warp = e >> 5, lane = e & 31;
  auto state = [&](int c) {
    return a.parts + ((static_cast<int64_t>(c) * 2 + (c == u.x)) * a.grp + r) * (D + 2);
  };
  // kAhead states at a time, everything asked for at once.
  float M = -CUDART_INF_F, L = 0.f, acc = 0.f;
  for (int c0 = u.x; c0 <= c1; c0 += kAhead) {
    const bool mine = e < kAhead && c0 + e <= c1;
    const float2 ml = mine ? *reinterpret_cast<const float2*>(state(c0 + e) + D)
                           : make_float2(-CUDART_INF_F, 0.f);
    float v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = c0 + k <= c1 ? state(c0 + k)[e] : 0.f;
    float mx = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[0][warp] = mx;
    __syncthreads();
    float top = M;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) top = fmaxf(top, red[0][w]);
    // (Equal, also where all are -inf: 1.)
    const float f = !mine ? 0.f : ml.x == top ? 1.f : ex2(ml.x - top);
    factor[e] = f;
    float sum = mine ? f * ml.y : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    const float old = M == top ? 1.f : ex2(M - top);
    L *= old;
    acc *= old;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) L += red[1][w];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k <= c1) acc += factor[k] * v[k];
    M = top;
    __syncthreads();
  }
  const int64_t row = static_cast<int64_t>(u.y) * a.Hq + u.z * a.grp + r;
  a.out[row * D + e] = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L * a.out_scale);
  if (e == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
}
template <int D>
__global__ void __launch_bounds__(D) decode_fp4_merge_kernel(const __grid_constant__ Fp4Args a) {
  pdl_wait();
  pdl_trigger();
  const int c1 = blockIdx.x;
  const int4 u = a.cut[c1];
  if (u.x < 0) return;
  if (c1 - u.x < 4)
    merge_cut<D, 4>(a, u, c1, blockIdx.y);
  else
    merge_cut<D, 40>(a, u, c1, blockIdx.y);
}

template <int D, int NT, bool LOGITS>
cudaError_t launch_t(const Fp4Args& a, int ctas, cudaStream_t stream) {
  using C = Fp4Cfg<D, NT>;
  auto kern = decode_fp4_kernel<D, NT, LOGITS>;
  static DeviceFlags smem_set;
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(ctas), dim3(kThreads), C::kSmemBytes, stream, a);
  if (e != cudaSuccess || a.whole || a.spans != nullptr) return e;
  return launch_pdl(decode_fp4_merge_kernel<D>, dim3(ctas, a.grp), dim3(D), 0, stream, a);
}
template <int D, int NT>
cudaError_t launch_n(const Fp4Args& a, int ctas, cudaStream_t stream) {
  return a.logits != nullptr ? launch_t<D, NT, true>(a, ctas, stream)
                             : launch_t<D, NT, false>(a, ctas, stream);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// CTAs that are resident at once, but no more than there are slices or units.
int decode_fp4_ctas(int N, int Hq, int Hkv, int max_seq_len, int sm_count) {
  const long long units = static_cast<long long>(N) * Hkv;
  const long long slices = units * ((static_cast<long long>(max_seq_len) + kSlice - 1) / kSlice);
    const long long most = static_cast<long long>(Hq / Hkv > 8 ? 1 : 2) * sm_count;
  return static_cast<int>(std::max(1LL, std::min(most, std::max(units, slices))));
}

// Units are not cut between CTAs where the longest is at most two slices for each warp:
// a second launch would cost more than the balance brings.
bool decode_fp4_whole(int max_seq_len) { return max_seq_len <= 2 * kSlice * kWarps; }
size_t decode_fp4_held(int ctas, int grp, int d) {
  return static_cast<size_t>(ctas) * kWarps * (grp > 8 ? 2 : 1) * (d / 16 + 1) * 512;
}

}  // namespace

Fp4Workspace decode_fp4_workspace(int N, int Hq, int Hkv, int d, int max_seq_len, bool sums,
                                  int sm_count) {
  Fp4Workspace w{};
  const size_t n = static_cast<size_t>(N);
  const int ctas = decode_fp4_ctas(N, Hq, Hkv, max_seq_len, sm_count);
  w.held = w.bytes;
  w.bytes += decode_fp4_held(ctas, Hq / Hkv, d);
  if (!decode_fp4_whole(max_seq_len)) {
    w.cut = w.bytes;
    w.bytes += static_cast<size_t>(ctas) * sizeof(int4);
    w.parts = w.bytes;
    w.bytes += up16(static_cast<size_t>(ctas) * 2 * (Hq / Hkv) * (d + 2) * 4);
  }
  if (sums) {
    w.spans = w.bytes;
    w.bytes += up16(n * Hkv * sizeof(int2));
    w.row_lse = w.bytes;
    w.bytes += up16(n * Hq * 4);
    w.logits = w.bytes;
    w.bytes += n * Hq * max_seq_len * 4;
  }
  return w;
}

cudaError_t launch_decode_fp4(const DecodeFp4Launch& n, cudaStream_t stream) {
  Fp4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(n.q);
  a.cache = static_cast<const uint8_t*>(n.cache);
  a.block_table = n.block_table;
  a.seq_lens = n.seq_lens;
  a.N = n.N;
  a.max_blocks = n.max_blocks;
  a.Hq = n.Hq;
  a.Hkv = n.Hkv;
  a.grp = n.Hq / n.Hkv;
  a.bs = n.bs;
  a.bs_log2 = block_size_log2(n.bs);
  a.num_blocks = n.num_blocks;
  a.whole = decode_fp4_whole(n.max_seq_len);
  a.positions = static_cast<int>(
      std::min(static_cast<long long>(n.max_blocks) * n.bs, INT_MAX - 1023LL));
  a.scale_log2 = n.scale * n.k_scale * kLog2e;
  a.out_scale = n.v_scale;
  const Fp4Workspace w =
      decode_fp4_workspace(n.N, n.Hq, n.Hkv, n.d, n.max_seq_len, n.scores != nullptr, n.sm_count);
  char* ws = static_cast<char*>(n.workspace);
  a.held = reinterpret_cast<float4*>(ws + w.held);
  if (!a.whole) {
    a.cut = reinterpret_cast<int4*>(ws + w.cut);
    a.parts = reinterpret_cast<float*>(ws + w.parts);
  }
  if (n.scores != nullptr) {
    a.spans = reinterpret_cast<int2*>(ws + w.spans);
    a.row_lse = reinterpret_cast<float*>(ws + w.row_lse);
    a.logits = reinterpret_cast<float*>(ws + w.logits);
    a.logit_tokens = n.max_seq_len;
  }
  a.out = static_cast<__nv_bfloat16*>(n.out);
  a.lse = n.lse;
  a.err = n.err;
  const int ctas = decode_fp4_ctas(n.N, n.Hq, n.Hkv, n.max_seq_len, n.sm_count);
  const bool wide = a.grp > 8;   // groups of 9 to 16 heads take two n-tiles
  cudaError_t e;
  if (n.d == 128)
    e = wide ? launch_n<128, 2>(a, ctas, stream) : launch_n<128, 1>(a, ctas, stream);
  else
    e = wide ? launch_n<64, 2>(a, ctas, stream) : launch_n<64, 1>(a, ctas, stream);
  if (e != cudaSuccess || n.scores == nullptr) return e;
  ScoresLaunch m{};
  m.parts = a.parts;
  m.spans = a.spans;
  m.row_lse = a.row_lse;
  m.out_scale = n.v_scale;
  m.logits = a.logits;
  m.logit_tokens = n.max_seq_len;
  m.seq_lens = n.seq_lens;
  m.positions = a.positions;
  m.N = n.N;
  m.Hq = n.Hq;
  m.Hkv = n.Hkv;
  m.d = n.d;
  m.max_seq_len = n.max_seq_len;
  m.scores = n.scores;
  m.score_tokens = n.score_tokens;
  m.out = n.out;
  m.lse = n.lse;
  m.err = n.err;
  return launch_decode_scores(m, stream);
}

}  // namespace pa
