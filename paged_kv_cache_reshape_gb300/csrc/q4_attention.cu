// Attention over pools held in 4 bits: one stream of pages per SM.
//
// Mathematics.  A code n in [0, 15] put into the low bits of an fp16 is the
// subnormal number n 2^-24, and one bit-and makes two of them at once, so
// codes become matrix operands without a conversion.  Nibbles 1 and 3 of a
// 16-bit half land four bits higher and are 16 times too large: for K the
// query's channels carry the 1/16, for V the output's.  With S^T = K Q^T
// (keys as the 16 rows of an MMA, up to 8 query rows as its columns) a
// group's scale is one multiply of its accumulator,
//   x_k = f sum_j s_kj (sum_c n_kjc q_c - 8 sum_c q_c),
// and the constant -8 sum q starts the accumulator.  For O^T = V^T P^T the
// scale goes to P: the product of a weight and its key's scale, rounded to
// fp16 once (the weight is kept as a pair of fp16, its rounding and the
// rest; with a rounding of its own the output of a long context was 10 to
// 20 % further off).  V's codes lose their 8 before they are multiplied,
// exactly: as a second MMA of the constant -8, or from the sums at the end,
// it left a small difference of large sums, which the tensor core cuts
// (4.7e-4 off instead of 2.8e-4 at 130,000 keys, 2.1e-4 of it the output's
// own rounding; the second MMA was also slower, 74.9 us against 72.5).
//
// Softmax in base 2 with a reference per row that moves only when a score
// passes it by 2^kSlack: weights are exp2(y - ref), where ref = max - k and
// 2^k holds the weights times V's scales near the top of fp16's range
// (below 2^15), whatever the scales are.
//
// Work.  A unit is up to 8 NT query rows (token x head) of a sequence and kv
// head, its keys steps of 16 tokens.  The steps of all units stand in one
// line, cut into one equal range per SM, so that few long and many short
// sequences both fill the GPU; a unit that a border cuts leaves partial
// results that a last kernel joins.  In a CTA one warp lays out the range
// in segments (whose steps, on which pages), and the others take its steps
// in turn: each copies its own steps ahead into stages of its own with
// cp.async, needs no one else, and keeps its own reference, sums and
// accumulators, joined through shared memory at the end of a unit.
//
// What bounds it.  Two sequences of 100,000 to 131,072 tokens, 64 query heads
// over 8 of 128: 262 MB in 75 us, 52 % of the copy rate; 64 sequences of 512 to
// 4,096, 32 over 8: 172 MB in 63 us, 40 %.  Neither memory nor the issue slots
// are full: about 330 instructions a step (the codes' masks, the scales, two
// MMA chains, the softmax) issue 47 to 55 % of the time with 11 or 12 warps of
// 162 registers, three to a scheduler, which wait for fixed latencies and at a
// unit's end for one another.  The steady state of long ranges reads at 64 to
// 68 % of the copy rate; about 15 us of a call are start, the units' ends and
// the join.  One user over 600 tokens: 15 us, the latency
// of two launches and a chain of 32 steps a range.
#include <algorithm>

#include "ptx.cuh"
#include "q4.h"
#include "step.h"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnit = 5.9604644775390625e-8f;  // 2^-24, what a code of 1 stands for
constexpr float kSlack = 4.f;
constexpr int kNoTiles = 0x7fffffff;  // stream_rows of a call without the tcgen05 kernel
constexpr int kSegSteps = 128;   // most steps of a segment
constexpr int kSegRing = 4;
constexpr int kMaxWarps = 20;
constexpr int kSmemLimit = 227 * 1024;
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;  // nibbles 0 and 1 of each half
constexpr uint32_t kEight = 0x00080008u, kEightHigh = 0x00800080u;  // 8 and 128, times 2^-24

// Part of a unit's steps in this CTA's range.
struct Seg {
  int n_steps;      // 0: no more segments
  int begin, last;  // whether a unit starts / ends here (for this CTA)
  int turn;         // the warp that takes the first steps
  int h;            // kv head
  int t0;           // packed row of the sequence's first token
  int row0, nrows;  // rows of the (sequence, kv head): token x group head
  int past;
  int part;         // slot of its partial results, -1: the whole unit is here
  int warps;        // warps that have had steps of the unit in this CTA (set with last)
  int unit_turn;    // the first of them
  int query;        // slot of its query rows
  int pad[2];
  // Each step: where its codes are in the pools (two words, bytes), its
  // first position, and what it is to the unit's rows (StepKind).
  int4 step[kSegSteps];
};
enum StepKind { kStepNone = 0, kStepPlain = 1, kStepMasked = 2 };  // no page or no row's; every row's; some

// A unit's query rows, laid out for the consumers.
template <int D, int NT>
struct QuerySlot {
  uint4 q[NT][D / 32][32];        // [group][lane]: B operands of S^T
  float c0[NT][D / 32][8];        // -8 2^-24 sum q of each row
  float f[NT][8];                 // of each row
};

struct Ctrl {
  Seg seg[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  long long scan[kMaxWarps];  // sums of the warps
  long long start_line;       // line position of the first sequence with work of this CTA
  int start_seq;
  int abort;
  float ml[kMaxWarps][kQ4Rows][2];  // [warp][row]: reference and sum
};

template <int D, int NT>
struct Cfg {
  // CTAs of an SM (with two, one streams on while the other joins a unit's
  // results, for one consumer warp less and twice the ranges: 256 units of
  // 2000 tokens 27 us against 32 at head_size 64, but 1024 of 4000 at
  // head_size 256 take 361 us against 324), and their consumer warps.  With the scheduling
  // warps they make 2 per scheduler of the SM (255 registers a thread), 3
  // (168) or 4 (128).
  static constexpr int kCtas = D == 64 ? 2 : 1;
  static constexpr int kWarps = (D == 256 || (D == 128 && NT == 2) ? 8 : D == 128 || NT == 2 ? 12 : 16) / kCtas - 1;
  static constexpr int kPer = D == 256 ? 1 : 2;        // steps that a warp takes at a time
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kGroups = D / 32;
  static constexpr int kHalf = 16 * (D / 2 + D / 16);  // K or V of a step: codes, then scales [D / 32][16]
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRowPitch = D + 4;              // floats of a row in the merge buffer
  static constexpr int kMergeBytes = kWarps * kRows * kRowPitch * 4;
  static constexpr int kTurn = kPer * kStage;
  static constexpr int kQueryBytes = kSegRing * (int)sizeof(QuerySlot<D, NT>);
  static constexpr int kFit = (kSmemLimit / kCtas - 1024 - (int)sizeof(Ctrl) - kMergeBytes - kQueryBytes) / (kWarps * kTurn);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;  // turns that a warp holds
  static constexpr int kSmem = kWarps * kStages * kTurn + kMergeBytes + kQueryBytes + (int)sizeof(Ctrl);
  static_assert(kStages >= 3, "stages");
  static constexpr int kVecs = kStage / 16, kLoads = (kVecs + 31) / 32;  // 16-byte copies of a step, per lane
};

// What a sequence adds to the line: row blocks x kv heads x the span of a
// unit, its steps and about as many more as its start, joining and output
// take the time of.  64 x 8 units of 500 to 4,100 tokens, heads of 128: 63 us
// with 36, 69 with 18, 66 with 72, 78 without; 200 x 8 of 200 to 2,500: 122,
// 132 and 124 us, heads of 64: 74, 81 and 78.  head_size 256, 200 x 4 of them:
// 105 us with 24, 114 with 12, 107 with 36; the window's 40 x 4: 64 with each.
template <int D>
constexpr int kUnitSpan = D == 256 ? 24 : 36;
struct SeqWork {
  int n, past, lo, first_steps, steps, blocks, span;
  long long len;
  // Steps of a unit that lie before y of its span.
  __device__ __forceinline__ int steps_before(int y) const { return (int)((long long)y * steps / span); }
};

template <int D>
__device__ __forceinline__ SeqWork seq_work(const Q4Params& p, int b, int rows, bool note) {
  SeqWork w;
  w.len = 0;
  const int c0 = p.g.cum[b], c1 = p.g.cum[b + 1];
  w.past = p.g.past[b];
  w.n = c1 - c0;
  w.steps = 0;
  if (c0 < 0 || c1 < c0 || c1 > p.g.T) {
    if (note) atomicOr(p.g.err, PA_DEVERR_CUM);
    return w;
  }
  if (w.n == 0) return w;
  if (w.past < 0 || (long long)w.past + w.n > p.g.max_kv) {
    if (note) atomicOr(p.g.err, w.past < 0 ? PA_DEVERR_PAST : PA_DEVERR_KV_BOUND);
    return w;
  }
  if ((long long)w.n * p.G > p.stream_rows) return w;  // the other kernel's
  w.lo = p.window > 0 ? max(0, w.past + 1 - p.window) & ~15 : 0;
  w.first_steps = (min(p.first, w.lo) + 15) / 16;
  w.steps = w.first_steps + (w.past + w.n - w.lo + 15) / 16;
  w.blocks = (int)(((long long)w.n * p.G + rows - 1) / rows);
  w.span = w.steps + kUnitSpan<D>;
  w.len = (long long)w.blocks * p.g.Hk * w.span;
  return w;
}

__device__ __forceinline__ int step_key(int i, int first_steps, int lo) {
  return i < first_steps ? 16 * i : lo + 16 * (i - first_steps);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Barrier of the consumer warps that tells every one whether any failed.
__device__ __forceinline__ bool consumers_any(int count, bool failed) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %1, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}\n"
      : "=r"(any)
      : "r"(count), "r"((int)failed)
      : "memory");
  return any != 0;
}

// D = A(16x16 f16, row) * B(16x8 f16, col) + C, C apart from D.
__device__ __forceinline__ void hmma_from(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 half2_floats(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2*>(&a)); }
// a's halves where the halves of w are not zero.
__device__ __forceinline__ uint32_t where_nonzero(uint32_t a, uint32_t w) {
  return a & __hne2_mask(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0)));
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t* w, const uint8_t* at) {
  if constexpr (N == 2) {
    *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 4) *reinterpret_cast<uint4*>(w + c) = *reinterpret_cast<const uint4*>(at + 4 * c);
  }
}

// A warp's share of a unit: the query's rows as operands, and what it has
// summed up.
template <int D, int NT>
struct Share {
  static constexpr int kGroups = D / 32;
  uint32_t q[NT][kGroups][4];     // B operands of S^T: row g, 8 channels of chunk t
  float c0[NT][kGroups][2];       // -8 2^-24 sum q of rows 2t, 2t + 1
  float f[NT][2];                 // from an accumulator to log2 units (or to twice the softcap's argument)
  int pos[NT][2], pos_max, lo_min;
  float ref[NT][2], lim[NT][2], l[NT][2];  // reference, score that moves it, sum
  float smax_lim;                 // largest scale of V that the references allow for
  float o[kGroups][2][NT][4];
};

// Scores of a step's 16 keys in log2 units: key ta (elements 0, 1) and
// ta + 2 (2, 3) of rows 2t and 2t + 1; what a row does not admit is -inf.
template <int D, int NT, bool CAP, bool M>
__device__ __forceinline__ void step_scores(const Q4Params& p, const Share<D, NT>& w, const uint8_t* at, int key0, float (&y)[NT][4]) {
  constexpr int kGroups = D / 32, kCodes = 16 * (D / 2);
  const int lane = threadIdx.x & 31, t = lane & 3, u4 = lane >> 3, ta = 4 * u4 + ((lane >> 2) & 1);
  uint32_t wa[kGroups], wb[kGroups];
  const uint8_t* chunk = at + ta * (D / 2) + (t ^ u4) * (D / 8);
  lds_words<kGroups>(wa, chunk);
  lds_words<kGroups>(wb, chunk + D);
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    const __half* sk = reinterpret_cast<const __half*>(at + kCodes + j * 32) + ta;
    const float2 s = make_float2(__half2float(sk[0]), __half2float(sk[2]));
    const uint32_t a8 = wa[j] >> 8, b8 = wb[j] >> 8;
    const uint32_t m0[4] = {wa[j] & kLow, wb[j] & kLow, wa[j] & kHigh, wb[j] & kHigh};
    const uint32_t m1[4] = {a8 & kLow, b8 & kLow, a8 & kHigh, b8 & kHigh};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float d[4];
      hmma_from(d, m0, w.q[nt][j][0], w.q[nt][j][1], w.c0[nt][j][0], w.c0[nt][j][1]);
      hmma16816(d, m1, w.q[nt][j][2], w.q[nt][j][3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[nt][e] = (e < 2 ? s.x : s.y) * d[e] + (j ? y[nt][e] : 0.f);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[nt][e] *= w.f[nt][e & 1];
      if constexpr (CAP) y[nt][e] = p.softcap * kLog2e * (1.f - 2.f * rcp(1.f + ex2(y[nt][e])));
      if constexpr (M) {
        const int key = key0 + ta + (e & 2), at_row = w.pos[nt][e & 1];
        if (!(key <= at_row && (p.window <= 0 || key > at_row - p.window || key < p.first))) y[nt][e] = -INFINITY;
      }
    }
}

// V's scales of keys 4t .. 4t + 3 of a step; of keys that no row admits
// (they may hold anything) zeros.
template <int D, int NT, bool M>
__device__ __forceinline__ void step_scales(const Q4Params& p, const Share<D, NT>& w, const uint8_t* at, int key0, uint2 (&sv)[D / 32]) {
  constexpr int kGroups = D / 32, kCodes = 16 * (D / 2), kHalf = 16 * (D / 2 + D / 16);
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    sv[j] = *reinterpret_cast<const uint2*>(at + kHalf + kCodes + j * 32 + 8 * t);
    if constexpr (M) {
      uint32_t keep[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = key0 + 4 * t + e;
        if (key <= w.pos_max && (key >= w.lo_min || key < p.first)) keep[e >> 1] |= e & 1 ? 0xffff0000u : 0x0000ffffu;
      }
      sv[j].x &= keep[0];
      sv[j].y &= keep[1];
    }
  }
}

// N steps, one stage behind the other; M: they have keys that some rows do
// not admit (N is 1 then), the first of them at key0.
template <int D, int NT, bool CAP, int N, bool M>
__device__ __forceinline__ void take_steps(const Q4Params& p, Share<D, NT>& w, const uint8_t* at, int key0) {
  constexpr int kGroups = D / 32, kHalf = 16 * (D / 2 + D / 16), kStage = 2 * kHalf;
  const int lane = threadIdx.x & 31, t = lane & 3, u4 = lane >> 3;
  const uint32_t sel_rows = lane & 4 ? 0x7632u : 0x5410u;  // of two words: the high or the low halves
  float y[N][NT][4];
#pragma unroll
  for (int h = 0; h < N; ++h) step_scores<D, NT, CAP, M>(p, w, at + h * kStage, key0, y[h]);
  bool moves = false;
  uint32_t bits = 0;
#pragma unroll
  for (int h = 0; h < N; ++h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) moves |= y[h][nt][e] > w.lim[nt][e & 1];
    uint2 sv[kGroups];
    step_scales<D, NT, M>(p, w, at + h * kStage, key0, sv);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) bits |= sv[j].x | sv[j].y;
  }
  // A scale of 2 or more (bit 14 of a half) may pass what the references
  // allow for; below that none does.
  float smax = 0.f;
  if (bits & 0x40004000u) {
#pragma unroll
    for (int h = 0; h < N; ++h) {
      uint2 sv[kGroups];
      step_scales<D, NT, M>(p, w, at + h * kStage, key0, sv);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const float2 a = half2_floats(sv[j].x), b = half2_floats(sv[j].y);
        smax = fmaxf(smax, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)));
      }
    }
    moves |= smax > w.smax_lim;
  }
  if (__any_sync(0xffffffffu, moves)) {
    // New references: these steps' largest scores and scales.
    float up[NT][2];
#pragma unroll
    for (int d = 16; d; d >>= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
    // 2^k times the largest scale, times 2^kSlack, stays below 2^15
    if (smax > w.smax_lim) w.smax_lim = ldexpf(1.f, min(ilogbf(smax), 24) + 1);
    const float k = 11.f - (float)ilogbf(w.smax_lim);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(y[0][nt][e], y[0][nt][e + 2]);
#pragma unroll
        for (int h = 1; h < N; ++h) top = fmaxf(top, fmaxf(y[h][nt][e], y[h][nt][e + 2]));
#pragma unroll
        for (int d = 16; d >= 4; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        // the old reference is that of a score lim - kSlack (none yet: lim = -inf)
        top = fmaxf(top, w.lim[nt][e] - kSlack);
        const bool none = top == -INFINITY;
        // (rounded up and the limit down: for scores past 2^24 a rounding may
        // be more than a weight's exponent has left)
        const float r1 = none ? 0.f : __fadd_ru(top, -k);
        up[nt][e] = w.lim[nt][e] == -INFINITY ? 0.f : ex2(w.ref[nt][e] - r1);
        w.ref[nt][e] = r1;
        w.lim[nt][e] = none ? -INFINITY : __fadd_rd(top, kSlack);
        w.l[nt][e] *= up[nt][e];
      }
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) w.o[j][a][nt][e] *= up[nt][e & 1];
  }
  uint32_t pb[N][NT][2], pr[N][NT][2];  // weights, and what their rounding left
#pragma unroll
  for (int h = 0; h < N; ++h)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ex2(y[h][nt][e] - w.ref[nt][e & 1]);
        // (an admitted key's weight is never 0, so that 0 says "not admitted" below)
        if (M && y[h][nt][e] > -INFINITY) x[e] = fmaxf(x[e], kUnit);
      }
      w.l[nt][0] += x[0] + x[2];
      w.l[nt][1] += x[1] + x[3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // keys 4t, 4t + 1 of row g; keys 4t + 2, 4t + 3
        const uint32_t both = pack_half2(x[2 * e], x[2 * e + 1]);
        const float2 back = half2_floats(both);
        pb[h][nt][e] = movmatrix_t(both);
        pr[h][nt][e] = movmatrix_t(pack_half2(x[2 * e] - back.x, x[2 * e + 1] - back.y));
      }
    }
#pragma unroll
  for (int h = 0; h < N; ++h) {
    const uint8_t* va = at + h * kStage + kHalf;
    uint32_t vw[4][kGroups];
    uint2 sv[kGroups];
#pragma unroll
    for (int i = 0; i < 4; ++i) lds_words<kGroups>(vw[i], va + (4 * t + i) * (D / 2) + (u4 ^ t) * (D / 8));
    step_scales<D, NT, M>(p, w, at + h * kStage, key0, sv);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      // nibble i of these halves: channel 32 j + 8 (g / 2) + 2 i + g % 2
      const uint32_t x0 = __byte_perm(vw[0][j], vw[1][j], sel_rows), x1 = __byte_perm(vw[2][j], vw[3][j], sel_rows);
      const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
      const uint32_t m0[4] = {hsub2_bits(x0 & kLow, kEight), hsub2_bits(x0 & kHigh, kEightHigh),
                              hsub2_bits(x1 & kLow, kEight), hsub2_bits(x1 & kHigh, kEightHigh)};
      const uint32_t m1[4] = {hsub2_bits(z0 & kLow, kEight), hsub2_bits(z0 & kHigh, kEightHigh),
                              hsub2_bits(z1 & kLow, kEight), hsub2_bits(z1 & kHigh, kEightHigh)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t b0 = hfma2_bits(pb[h][nt][0], sv[j].x, hmul2_bits(pr[h][nt][0], sv[j].x));
        uint32_t b1 = hfma2_bits(pb[h][nt][1], sv[j].y, hmul2_bits(pr[h][nt][1], sv[j].y));
        if constexpr (M) {  // 0 times a NaN scale is 0 for a key that the row does not admit
          b0 = where_nonzero(b0, pb[h][nt][0]);
          b1 = where_nonzero(b1, pb[h][nt][1]);
        }
        hmma16816(w.o[j][0][nt], m0, b0, b1);
        hmma16816(w.o[j][1][nt], m1, b0, b1);
      }
    }
  }
}

// Query rows as B operands: lane (row g, chunk t) of each group, times a
// power of two that brings the row's largest value near the top of fp16 (so
// that the conversion loses nothing), and a 16th of that where the code is
// in a high nibble.  One warp.
template <int D, int NT, bool CAP>
__device__ __forceinline__ void lay_out_query(const Q4Params& p, int t0, int h, int row0, int nrows, QuerySlot<D, NT>& to) {
  constexpr int kGroups = D / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    uint4 raw[kGroups];
    const bool have = r < nrows;
    const int rho = row0 + (have ? r : 0), tok = rho / p.G;
    const __half* src = p.query + ((size_t)(t0 + tok) * p.H + h * p.G + (rho - tok * p.G)) * D + 8 * t;
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
      raw[j] = have ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0, 0, 0, 0);
    auto values = [&](int j, float* x) {
      const uint32_t word[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.bf16) {
          x[2 * e] = __uint_as_float(word[e] << 16);
          x[2 * e + 1] = __uint_as_float(word[e] & 0xffff0000u);
        } else {
          const float2 h2 = half2_floats(word[e]);
          x[2 * e] = h2.x;
          x[2 * e + 1] = h2.y;
        }
      }
    };
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      float x[8];
      values(j, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^up in two factors (a bfloat16 row may need more than 2^127)
    const int up = top > 0.f && top < INFINITY ? 14 - ilogbf(top) : 0;
    const float up0 = __int_as_float((127 + up / 2) << 23), up1 = __int_as_float((127 + up - up / 2) << 23);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      float x[8], s = 0.f;
      values(j, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = x[e] * up0 * up1;
        s += x[e];
      }
      to.q[nt][j][lane] = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2] * 0.0625f, x[3] * 0.0625f),
                                     pack_half2(x[4], x[5]), pack_half2(x[6] * 0.0625f, x[7] * 0.0625f));
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (t == 0) to.c0[nt][j][g] = s * (-8.f * kUnit);
    }
    // (finite where the scores are: the largest queries' exponent and the codes'
    // 2^24 together may pass 2^127, and scores of 0 have to stay 0)
    const float f = ldexpf(CAP ? 2.f * kLog2e * p.scale / p.softcap : p.scale * kLog2e, 24 - up);
    if (t == 0) to.f[nt][g] = fminf(f, 3.402823466e38f);
  }
}

template <int D, int NT, bool CAP>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtas) q4_stream_kernel(const __grid_constant__ Q4Params p) {
  using C = Cfg<D, NT>;
  constexpr int kGroups = C::kGroups, NW = C::kWarps, S = C::kStages, PER = C::kPer;
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + NW * S * C::kTurn);
  auto* queries = reinterpret_cast<QuerySlot<D, NT>*>(smem + NW * S * C::kTurn + C::kMergeBytes);
  Ctrl* ctl = reinterpret_cast<Ctrl*>(smem + NW * S * C::kTurn + C::kMergeBytes + C::kQueryBytes);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&ctl->seg_full[i], 1);
      mbar_init(&ctl->seg_empty[i], NW);
    }
    ctl->abort = 0;
    ctl->start_seq = 0x7fffffff;
    fence_mbar_init();
  }
  griddep_wait();
  // The next kernel's CTAs may come as soon as there is room.  Not before the
  // end where it is the tcgen05 kernel at head_size 64: that one leaves 90 KB
  // of an SM to its L1, but only if it starts on an empty one; among this
  // kernel's CTAs it keeps their 28 KB (32 x 260 rows after 3,000 tokens 251 us
  // instead of 229, up to 800 rows a sequence 281 instead of 249).  At 128 it
  // needs all shared memory itself, and the end is worth -2 % to +2 %.
  if (D != 64 || p.stream_rows == kNoTiles) griddep_launch_dependents();

  // The line: every thread sums a share of the sequences, and the one whose
  // share holds the start of this CTA's range finds the sequence.
  const int per = (p.g.batch + C::kThreads - 1) / C::kThreads;
  const int s0 = min(p.g.batch, (int)threadIdx.x * per), s1 = min(p.g.batch, s0 + per);
  long long sum = 0;
  for (int b = s0; b < s1; ++b) sum += seq_work<D>(p, b, C::kRows, blockIdx.x == 0).len;
  if (blockIdx.x == 0 && threadIdx.x == 0 && (p.g.cum[0] != 0 || p.g.cum[p.g.batch] > p.g.T))
    atomicOr(p.g.err, PA_DEVERR_CUM);
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) ctl->scan[warp] = incl;
  __syncthreads();
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w <= NW; ++w) {
    const long long s = ctl->scan[w];
    if (w < warp) before += s;
    total += s;
  }
  // (None but those behind the last is empty, and none shorter than kLeast:
  // the warps take that many steps at once anyway, and a unit in fewer pieces
  // is joined sooner.  One user over 600 tokens: 19 us with ranges of 4, 15.5
  // with 32, 17.8 with 96; over 4,000: 16.8 with 32, 19.2 with 16, 20.2 with
  // 64, head_size 256 23.1, 23.9 and 24.7.)
  constexpr int kLeast = 32;
  const long long ranges = min((long long)gridDim.x, (total + kLeast - 1) / kLeast), me = min((long long)blockIdx.x, ranges);
  const long long r0 = ranges ? total * me / ranges : 0, r1 = me < ranges ? total * (me + 1) / ranges : r0;
  if (sum > 0 && r0 < r1 && r0 >= before && r0 < before + sum) {
    long long at = before;
    for (int b = s0; b < s1; ++b) {
      const long long len = seq_work<D>(p, b, C::kRows, false).len;
      if (r0 < at + len) {
        ctl->start_seq = b;
        ctl->start_line = at;
        break;
      }
      at += len;
    }
  }
  __syncthreads();

  if (warp == NW) {
    // ----------------------------------------------------------- scheduler
    Q4Cut cut;
    cut.pieces = 0;
    const int run = q4_run_bytes(p.g.bs, D);
    long long x = r0, line = ctl->start_line;
    uint32_t n_segs = 0, n_units = 0;
    int b = ctl->start_seq, turn = 0;
    bool ok = true;
    while (ok && x < r1 && b < p.g.batch) {
      const SeqWork w = seq_work<D>(p, b, C::kRows, false);
      if (x >= line + w.len) {
        line += w.len;
        ++b;
        continue;
      }
      const int* row = p.g.block_table + (size_t)b * p.g.MB;
      const int t0 = p.g.cum[b];
      while (ok && x < r1 && x < line + w.len) {
        const long long in = x - line;
        const int idx = (int)(in / w.span), y0 = (int)(in - (long long)idx * w.span);
        const int y1 = (int)min((long long)w.span, y0 + (r1 - x));  // the unit's span here
        const int i0 = w.steps_before(y0), n = w.steps_before(y1) - i0;
        const int blk = idx / p.g.Hk, h = idx - blk * p.g.Hk, unit_turn = turn;
        const int row0 = blk * C::kRows, nrows = (int)min((long long)C::kRows, (long long)w.n * p.G - row0);
        const int pos_min = w.past + row0 / p.G, pos_max = w.past + (row0 + nrows - 1) / p.G;
        const int lo_min = p.window > 0 ? max(0, pos_min + 1 - p.window) : 0;
        const int lo_max = p.window > 0 ? max(0, pos_max + 1 - p.window) : 0;
        const bool from_start = y0 == 0, to_end = y1 == w.span;
        const int part = from_start && to_end ? -1 : 2 * (int)blockIdx.x + (from_start ? 1 : 0);
        if (n == 0 && lane < C::kRows)  // a piece without a step
          p.part_ml[(size_t)part * C::kRows + lane] = make_float2(-INFINITY, 0.f);
        for (int k0 = 0; ok && k0 < n; k0 += kSegSteps) {
          Seg& s = ctl->seg[n_segs % kSegRing];
          int good = 1;
          if (lane == 0)
            good = wait_or_abort(&ctl->seg_empty[n_segs % kSegRing], ((n_segs / kSegRing) & 1) ^ 1, abort, p.g.err,
                                 p.err_site, kSiteQ4 | 1);
          ok = __shfl_sync(0xffffffffu, good, 0);
          if (!ok) break;
          const int m = min(kSegSteps, n - k0);
          if (k0 == 0) lay_out_query<D, NT, CAP>(p, t0, h, row0, nrows, queries[n_units % kSegRing]);
          for (int k = lane; k < m; k += 32) {
            const int key = step_key(i0 + k0 + k, w.first_steps, w.lo);
            const int page = row[key >> p.g.log_bs];
            const bool held = page >= 0 && page < p.g.NB;
            if (!held && page != -1) atomicOr(p.g.err, PA_DEVERR_BLOCK_ID);
            const long long at = ((long long)page * p.g.Hk + h) * run + (long long)(key & (p.g.bs - 1)) * (D / 2);
            const bool any = held && key <= pos_max && (key + 15 >= lo_min || key < p.first);
            const bool all = key + 15 <= pos_min && (key >= lo_max || key + 16 <= p.first);
            s.step[k] = make_int4((int)at, (int)(at >> 32), key, !any ? kStepNone : all ? kStepPlain : kStepMasked);
          }
          if (lane == 0) {
            s.n_steps = m;
            s.begin = k0 == 0;
            s.last = k0 + m == n;
            s.turn = turn;
            s.h = h;
            s.t0 = t0;
            s.row0 = row0;
            s.nrows = nrows;
            s.past = w.past;
            s.part = part;
            s.warps = min((n + PER - 1) / PER, NW);
            s.unit_turn = unit_turn;
            s.query = n_units % kSegRing;
          }
          turn = (turn + (m + PER - 1) / PER) % NW;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->seg_full[n_segs % kSegRing]);
          ++n_segs;
        }
        if (from_start && !to_end) {
          const long long last = x + w.span - 1;  // of the unit; the range that holds it
          cut.pieces = (int)(((last + 1) * ranges - 1) / total) - (int)blockIdx.x + 1;
          cut.t0 = t0;
          cut.row0 = row0;
          cut.nrows = nrows;
          cut.h = h;
        }
        x += y1 - y0;
        if (n) ++n_units;
      }
    }
    if (lane == 0) {
      p.cuts[blockIdx.x] = cut;
      const uint32_t s = n_segs % kSegRing;
      if (ok && wait_or_abort(&ctl->seg_empty[s], ((n_segs / kSegRing) & 1) ^ 1, abort, p.g.err, p.err_site, kSiteQ4 | 1)) {
        ctl->seg[s].n_steps = 0;
        mbar_arrive(&ctl->seg_full[s]);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3, u4 = g >> 1, odd = g & 1;
  uint8_t* stages = smem + warp * S * C::kTurn;
  // A step's copies: codes of K, scales of K, codes of V, scales of V, as
  // 16-byte vectors dealt to the lanes.  Two of a lane's vectors lie at a
  // border of these parts; for them, the offset from the step's codes (of K
  // or V) and how it moves with the step's row in its page.
  constexpr int kCodeVecs = D / 2, kHalfVecs = C::kHalf / 16;
  constexpr int kMix[2] = {kCodeVecs / 32, C::kLoads - 1};
  int mix_off[2], mix_mul[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int c = lane + 32 * kMix[m], cc = c >= kHalfVecs ? c - kHalfVecs : c, sc = cc - kCodeVecs;
    mix_off[m] = cc < kCodeVecs ? cc * 16 : p.g.bs * (D / 2) + (sc >> 1) * p.g.bs * 2 + (sc & 1) * 16;
    mix_mul[m] = cc < kCodeVecs ? 0 : 2 - D / 2;
  }
  auto first_step = [&](const Seg& s) { return PER * (warp >= s.turn ? warp - s.turn : warp - s.turn + NW); };

  // The loading side: up to S - 1 steps ahead of the computing side, over
  // segments.  Looking ahead waits for nothing (a segment that is not there
  // yet may need this warp to let go of one first); a step that is due does.
  uint32_t n_seg = 0, l_seg = 0;
  int l_k = 0, l_n = -1;  // next step of segment l_seg and their number; -1: not looked at yet
  int l_stage = 0, ahead = 0;
  bool l_end = false, failed = false;
  auto load_next = [&](bool due) -> bool {
    while (!l_end && l_k >= l_n) {
      if (l_n >= 0) {
        if (l_seg - n_seg == kSegRing - 1) return false;
        ++l_seg;
        l_n = -1;
      }
      const uint32_t at = l_seg % kSegRing, parity = (l_seg / kSegRing) & 1;
      if (due) {
        if (!warp_wait(&ctl->seg_full[at], parity, abort, p.g.err, p.err_site, kSiteQ4 | 2)) {
          failed = l_end = true;
          break;
        }
      } else if (!__all_sync(0xffffffffu, mbar_test_wait(&ctl->seg_full[at], parity))) {
        l_k = 0;
        return false;
      }
      l_n = ctl->seg[at].n_steps;
      l_k = first_step(ctl->seg[at]);
      l_end = l_n == 0;
    }
    if (l_end) return false;
    const Seg& from = ctl->seg[l_seg % kSegRing];
#pragma unroll
    for (int h = 0; h < PER; ++h) {
      const int4 rec = l_k + h < l_n ? from.step[l_k + h] : make_int4(0, 0, 0, kStepNone);
      if (rec.w == kStepNone) continue;
      const int r = rec.z & (p.g.bs - 1);
      const long long at = (long long)(((unsigned long long)(unsigned)rec.y << 32) | (unsigned)rec.x);
      const uint8_t *k_at = p.key_cache + at, *v_at = p.value_cache + at;
      const uint32_t dst = smem_u32(stages + l_stage * C::kTurn + h * C::kStage) + lane * 16;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        if (32 * (i + 1) <= kCodeVecs) {
          cp_async16(dst + 512 * i, k_at + lane * 16 + 512 * i);
        } else if (32 * i >= kHalfVecs && 32 * (i + 1) <= kHalfVecs + kCodeVecs) {
          cp_async16(dst + 512 * i, v_at + lane * 16 + (512 * i - C::kHalf));
        } else {
          const int m = i == kMix[0] ? 0 : 1, c = lane + 32 * i;
          if (c < C::kVecs) cp_async16(dst + 512 * i, (c >= kHalfVecs ? v_at : k_at) + (mix_off[m] + r * mix_mul[m]));
        }
      }
    }
    cp_async_commit();
    l_k += PER * NW;
    l_stage = l_stage + 1 == S ? 0 : l_stage + 1;
    ++ahead;
    return true;
  };

  Share<D, NT> w;
  int stage = 0;
  for (;; ++n_seg) {
    const uint32_t is = n_seg % kSegRing;
    const Seg& u = ctl->seg[is];
    if (!warp_wait(&ctl->seg_full[is], (n_seg / kSegRing) & 1, abort, p.g.err, p.err_site, kSiteQ4 | 3)) failed = true;
    const bool end = failed || u.n_steps == 0;
    if (!end) {
      while (ahead < S - 1 && load_next(false)) {
      }
    }
    const int k_first = end ? 0 : first_step(u);
    if (!end && u.begin) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w.ref[nt][e] = 0.f;
          w.lim[nt][e] = -INFINITY;
          w.l[nt][e] = 0.f;
        }
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[j][a][nt][e] = 0.f;
      w.smax_lim = 2.f;
      const QuerySlot<D, NT>& from = queries[u.query];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          const uint4 x = from.q[nt][j][lane];
          w.q[nt][j][0] = x.x;
          w.q[nt][j][1] = x.y;
          w.q[nt][j][2] = x.z;
          w.q[nt][j][3] = x.w;
          const float2 c = *reinterpret_cast<const float2*>(&from.c0[nt][j][2 * t]);
          w.c0[nt][j][0] = c.x;
          w.c0[nt][j][1] = c.y;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w.f[nt][e] = from.f[nt][2 * t + e];
          w.pos[nt][e] = u.past + (u.row0 + min(nt * 8 + 2 * t + e, u.nrows - 1)) / p.G;
        }
      }
      w.pos_max = u.past + (u.row0 + u.nrows - 1) / p.G;
      w.lo_min = p.window > 0 ? max(0, u.past + u.row0 / p.G + 1 - p.window) : 0;
    }

    const int n_steps = end ? 0 : u.n_steps;
    for (int k = k_first; k < n_steps; k += PER * NW) {
      if (ahead == 0 && !load_next(true)) break;
      if (ahead == S - 1) cp_async_wait<S - 2>();
      else cp_async_wait<0>();
      __syncwarp();
      const uint8_t* at = stages + stage * C::kTurn;
      int kind[PER], key0[PER];
      bool plain = true;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        kind[h] = k + h < n_steps ? u.step[k + h].w : kStepNone;
        key0[h] = k + h < n_steps ? u.step[k + h].z : 0;
        plain &= kind[h] == kStepPlain;
      }
      if (plain) {
        take_steps<D, NT, CAP, PER, false>(p, w, at, 0);
      } else {
#pragma unroll 1
        for (int h = 0; h < PER; ++h)
          if (kind[h] != kStepNone) take_steps<D, NT, CAP, 1, true>(p, w, at + h * C::kStage, key0[h]);
      }
      __syncwarp();
      stage = stage + 1 == S ? 0 : stage + 1;
      --ahead;
      while (ahead < S - 1 && load_next(false)) {
      }
    }

    if (end || failed || u.last) {
      if (!end && !failed && (u.warps == NW || (warp - u.unit_turn + NW) % NW < u.warps)) {
        // This warp's results: the sums over its lanes, and the accumulators
        // as [row][channel], in units of 2^-24.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float s = w.l[nt][e];
#pragma unroll
            for (int d = 16; d >= 4; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (g == 0) {
              ctl->ml[warp][nt * 8 + 2 * t + e][0] = w.lim[nt][e] == -INFINITY && s == 0.f ? -INFINITY : w.ref[nt][e];
              ctl->ml[warp][nt * 8 + 2 * t + e][1] = s;
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
              for (int a = 0; a < 2; ++a) {
                float* to = merge + (warp * C::kRows + nt * 8 + 2 * t + e) * C::kRowPitch + 32 * j + 8 * u4 + odd + 4 * a;
                to[0] = w.o[j][a][nt][e];
                to[2] = w.o[j][a][nt][e + 2] * 0.0625f;
              }
          }
      }
      if (consumers_any(NW * 32, failed) || end) {
        cp_async_wait<0>();
        return;
      }
      // Join the warps' results: a thread takes 4 channels of a row.
      const int n_parts = u.warps;
      for (int x = threadIdx.x; x < u.nrows * (D / 4); x += NW * 32) {
        const int r = x / (D / 4), c = (x - r * (D / 4)) * 4;
        float top = -INFINITY, ref[NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const int k = i - u.unit_turn + (i < u.unit_turn ? NW : 0);
          ref[i] = k < n_parts ? ctl->ml[i][r][0] : -INFINITY;
          top = fmaxf(top, ref[i]);
        }
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          if (ref[i] == -INFINITY) continue;  // no steps, or no admitted key
          const float up = ex2(ref[i] - top);
          const float4 a = *reinterpret_cast<const float4*>(merge + (i * C::kRows + r) * C::kRowPitch + c);
          sum += up * ctl->ml[i][r][1];
          v.x += up * a.x;
          v.y += up * a.y;
          v.z += up * a.z;
          v.w += up * a.w;
        }
        if (u.part >= 0) {
          const size_t at = (size_t)u.part * C::kRows + r;
          *reinterpret_cast<float4*>(p.part_o + at * D + c) = v;
          if (c == 0) p.part_ml[at] = make_float2(top, sum);
        } else {
          const int rho = u.row0 + r, tok = rho / p.G, h = u.h * p.G + rho - tok * p.G;
          q4_store(p, u.t0 + tok, h, D, c, v, top, sum, 1.f / kUnit);
        }
      }
      consumers_any(NW * 32, false);  // the buffers are free again
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->seg_empty[is]);
  }
}

// Joins the pieces of the units that the ranges cut: a block per range and
// 256 / (D / 4) rows, the
// first piece in the range's second place, later ones in the first place of
// the ranges that follow.
template <int D, int ROWS>
__device__ __forceinline__ void join_stream(const Q4Params& p, int range, int group) {
  constexpr int kRowThreads = D / 4;
  const Q4Cut cut = p.cuts[range];
  const int r = group * (256 / kRowThreads) + threadIdx.x / kRowThreads, c = threadIdx.x % kRowThreads * 4;
  if (cut.pieces == 0 || r >= cut.nrows) return;
  auto at = [&](int k) { return (size_t)(2 * (range + k) + (k == 0)) * ROWS + r; };
  float top = -INFINITY;
  for (int k = 0; k < cut.pieces; ++k) top = fmaxf(top, p.part_ml[at(k)].x);
  const bool none = top == -INFINITY;
  float sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < cut.pieces; ++k) {
    const float2 ml = p.part_ml[at(k)];
    const float4 a = *reinterpret_cast<const float4*>(p.part_o + at(k) * D + c);
    const float up = none ? 0.f : ex2(ml.x - top);
    if (ml.x == -INFINITY) continue;  // (what it holds may be anything)
    sum += up * ml.y;
    v.x += up * a.x;
    v.y += up * a.y;
    v.z += up * a.z;
    v.w += up * a.w;
  }
  const int rho = cut.row0 + r, tok = rho / p.G, h = cut.h * p.G + rho - tok * p.G;
  q4_store(p, cut.t0 + tok, h, D, c, v, top, sum, 1.f / kUnit);
}

// The same for the tcgen05 kernel's pieces, a block per range and 16
// channels; neighbouring threads take neighbouring rows, as the pieces lie.
constexpr int kJoinChannels = 16;
template <int D>
__device__ __forceinline__ void join_tiles(const Q4Params& p, int range, int group) {
  const Q4Cut cut = p.tile_cuts[range];
  const int r = threadIdx.x;
  if (cut.pieces == 0 || r >= cut.nrows) return;
  auto part = [&](int k) { return (size_t)(2 * (range + k) + (k == 0)); };
  float top = -INFINITY;
  for (int k = 0; k < cut.pieces; ++k) top = fmaxf(top, p.tile_ml[part(k) * kQ4TileRows + r].x);
  float sum = 0.f;
  float4 v[kJoinChannels / 4];
#pragma unroll
  for (int q = 0; q < kJoinChannels / 4; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < cut.pieces && top != -INFINITY; ++k) {
    const float2 ml = p.tile_ml[part(k) * kQ4TileRows + r];
    if (ml.x == -INFINITY) continue;
    const float up = ex2(ml.x - top);
    sum += up * ml.y;
    const float4* o = reinterpret_cast<const float4*>(p.tile_o) + (part(k) * (D / 4) + group * (kJoinChannels / 4)) * kQ4TileRows + r;
#pragma unroll
    for (int q = 0; q < kJoinChannels / 4; ++q) {
      const float4 a = o[(size_t)q * kQ4TileRows];
      v[q].x += up * a.x;
      v[q].y += up * a.y;
      v[q].z += up * a.z;
      v[q].w += up * a.w;
    }
  }
  const int rho = cut.row0 + r, tok = rho / p.G, h = cut.h * p.G + rho - tok * p.G;
#pragma unroll
  for (int q = 0; q < kJoinChannels / 4; ++q)
    q4_store(p, cut.t0 + tok, h, D, group * kJoinChannels + 4 * q, v[q], top, sum, 8.f);
}

// Blocks of the stream's joins, then of the tiles' (none where those did not
// run): one launch for both, since an empty one costs 2 to 3 us.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) q4_join_kernel(const __grid_constant__ Q4Params p, int ranges) {
  constexpr int kGroups = (ROWS * (D / 4) + 255) / 256;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x - ranges * kGroups;
  if (b < 0) {
    join_stream<D, ROWS>(p, blockIdx.x % ranges, blockIdx.x / ranges);
  } else if constexpr (ROWS == 16) {  // (as tiles ask for units of 16 rows)
    join_tiles<D>(p, b % p.num_sms, b / p.num_sms);
  }
}

template <int D, int NT>
cudaError_t launch(const Q4Params& p, bool tiles, bool configure, cudaStream_t s) {
  using C = Cfg<D, NT>;
  auto kernel = p.softcap > 0.f ? q4_stream_kernel<D, NT, true> : q4_stream_kernel<D, NT, false>;
  if (configure) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  const int ranges = p.num_sms * C::kCtas;
  cudaError_t e = launch_pdl(kernel, dim3(ranges), C::kThreads, C::kSmem, s, p);
  if (e == cudaSuccess && tiles) e = launch_q4_tile(p, s);
  if (e != cudaSuccess) return e;
  const int blocks = ranges * ((C::kRows * (D / 4) + 255) / 256) + (tiles ? p.num_sms * (D / kJoinChannels) : 0);
  return launch_pdl(q4_join_kernel<D, C::kRows>, dim3(blocks), 256, 0, s, p, ranges);
}

cudaError_t dispatch(const Q4Params& p, int nt, bool tiles, bool configure, cudaStream_t s) {
  switch (p.g.D * 4 + nt) {
    case 64 * 4 + 1: return launch<64, 1>(p, tiles, configure, s);
    case 64 * 4 + 2: return launch<64, 2>(p, tiles, configure, s);
    case 128 * 4 + 1: return launch<128, 1>(p, tiles, configure, s);
    case 128 * 4 + 2: return launch<128, 2>(p, tiles, configure, s);
    default: return launch<256, 1>(p, tiles, configure, s);
  }
}

}  // namespace

cudaError_t q4_configure(int D, float softcap) {
  Q4Params p{};
  p.g.D = D;
  p.softcap = softcap;
  cudaError_t e = dispatch(p, 1, false, true, nullptr);
  if (e == cudaSuccess && D < 256) e = dispatch(p, 2, false, true, nullptr);
  if (e == cudaSuccess && D < 256) e = q4_tile_configure(D, softcap);
  return e;
}

cudaError_t launch_q4_attention(const Q4Params& p0, cudaStream_t s) {
  Q4Params p = p0;
  // 8 rows a unit where a sequence's rows are that few (one token each of up
  // to 8 heads a kv head), else 16: the codes of a key are made into operands
  // once for all rows of a unit.  head_size 256 has registers for 8.
  // (As a rule: with T <= batch most sequences have a token each.  A chunk among
  // empty slots is right too, but reads its keys once for 8 rows; the host cannot
  // tell, and a launch that serves no sequence would cost each such call 6 us.)
  const bool single = p.g.T <= p.g.batch && p.G <= 8;
  const int nt = p.g.D < 256 && !single ? 2 : 1;
  // Sequences of more rows than two such units go to the tcgen05 kernel, whose
  // time hardly depends on their number up to a tile's 128 (32 sequences of
  // 3000 tokens, 8 kv heads of 128: 32 rows take 126 us here and 136 there, 36
  // rows 167 and 133).  Where most have fewer, a sequence of up to three units
  // is better left here, for the few that there are (1 to 9 tokens of 4 heads
  // after up to 3000: 79 us with three, 95 with two; heads of 64 48 and 59; 64
  // sequences of 1 to 6 tokens of 8 heads 78 and 101; rows of 36 in every
  // sequence would take 166 and 133, heads of 64 94 and 82).  The mean decides,
  // as the host knows no sequence's rows: above 28 calls of 1 to 12 tokens of
  // 4 heads (mean 28.5) lose 90 -> 103, but ones of equal rows gain as much.
  const long long rows = (long long)p.g.T * p.G;
  const int stream_rows = rows <= 28LL * p.g.batch ? 48 : 32;
  const bool tiles = nt == 2 && rows > stream_rows;
  p.stream_rows = tiles ? stream_rows : kNoTiles;
  return dispatch(p, nt, tiles, false, s);
}

}  // namespace pa
