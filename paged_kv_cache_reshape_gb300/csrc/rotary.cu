// Rotary embedding at explicit positions.
//
// Pair i of a row at position p turns by a = 2 pi frac(p f_i / 2 pi).  The
// frequency is held as step_i = f_i / (2 pi) in 2^-64 turns, so the phase is
// the wrapping 64-bit product p * step_i: exact modulo one turn for every p
// (also negative), where a 32-bit angle p * f_i loses 0.06 radians at a
// million positions.  The top 32 bits of the phase, as a signed fraction of a
// half turn, go to sincospif (angle error 2^-25 of a half turn); then
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
// in fp32 with one rounding to the output type.  The gradient of y with
// respect to x is the same map with -a (sin_sign -1).
//
// Bound by memory: every row is read and written once, and a token's R/2
// cosines and sines are computed once per warp and shared by all its heads
// through shared memory.  A warp takes one token and a share of its items, an
// item being one 16-byte vector, or the two of a pair of halves; the share
// shrinks when tokens are few, so that a short draft still fills several warps
// with independent loads.  A lane loads a batch of items at a time, the first
// one before it looks up the token's position and slot, whose chain of
// dependent loads would otherwise come before the first row is asked for.
// Where a head's items divide a warp (FIXED: the whole head rotates, a power
// of two of vectors), a lane meets the same pairs in every head and keeps
// their cosines and sines in registers; reading them from shared memory for
// every item took half the kernel's time.
//
// Measured (one GB300, 6780 GB/s copied): 16385 rows of 32 + 8 heads of 128,
// 64 channels interleaved, 54 us = 6.2 TB/s; 64 sequences of up to 64 drafts
// of 64 + 8 heads into the pool (89 MB), 25 us = 3.6 TB/s, where a plain copy
// of the same bytes takes 20.7 us: start, owner lookup and the tail of one
// wave.  Loading the next batch while the last one is stored took registers
// that cost more loads in flight than it gained (64 us for the 54).
//
// Pool mode: K (rotated) and V (copied) rows go to slot past_b + j through
// the block table, the same slot rule as the plain cache write.
#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "step.h"
#include "tree.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxPairs = 256;  // R / 2 for R <= 512
constexpr int kBatch = 4;       // items a lane loads before it stores
constexpr int kWantWarps = 1536;  // about ten per SM; tokens are cut into shares below that

template <int DT>
struct Elem {
  using T = uint16_t;
  static constexpr int kVec = 8;  // elements of a 16-byte vector
};
template <>
struct Elem<PA_ROTARY_FP32> {
  using T = float;
  static constexpr int kVec = 4;
};

template <int DT>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (DT == PA_ROTARY_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else if constexpr (DT == PA_ROTARY_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
      f[2 * i] = __low2float(h);
      f[2 * i + 1] = __high2float(h);
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float* f) {
  if constexpr (DT == PA_ROTARY_FP32)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(pack2<DT == PA_ROTARY_BF16>(f[0], f[1]), pack2<DT == PA_ROTARY_BF16>(f[2], f[3]),
                      pack2<DT == PA_ROTARY_BF16>(f[4], f[5]), pack2<DT == PA_ROTARY_BF16>(f[6], f[7]));
}

// The items of a token stand in one line: those of its Q heads, of its K
// heads, then V's plain vectors.
struct Line {
  int per_head;        // items of a rotated head
  int log_head;        // log2 of them (FIXED)
  float inv_head;
  int nq, nk, nv;      // items of Q, K, V
};

struct Item {
  int part;            // 0 Q, 1 K, 2 V
  int at, mate, pair;  // element offset, that of the partner vector (half layout), first pair (-1: copied)
};

template <int DT, bool INTER, bool FIXED>
__device__ __forceinline__ Item item_of(int i, const Line& n, const RotaryParams& p) {
  constexpr int V = Elem<DT>::kVec;
  Item it;
  it.mate = it.pair = -1;
  it.part = i < n.nq ? 0 : i < n.nq + n.nk ? 1 : 2;
  if (it.part == 2) {
    it.at = (i - n.nq - n.nk) * V;
    return it;
  }
  if (it.part == 1) i -= n.nq;
  const int h = FIXED ? i >> n.log_head : (int)(((float)i + 0.5f) * n.inv_head);  // exact below 2^20 items
  const int c = i - h * n.per_head;
  if constexpr (INTER) {
    const int ch = c * V;
    it.at = h * p.D + ch;
    if (ch >= p.off && ch < p.off + p.R) it.pair = (ch - p.off) / 2;
  } else {
    const int pairs = p.R / 2 / V;
    if (c < pairs) {
      it.at = h * p.D + p.off + c * V;
      it.mate = it.at + p.R / 2;
      it.pair = c * V;
    } else {
      const int ch = (c - pairs) * V;
      it.at = h * p.D + (ch < p.off ? ch : ch + p.R);
    }
  }
  return it;
}

template <int DT, bool INTER, bool FIXED>
__global__ void __launch_bounds__(kWarps * 32) rotary_kernel(const RotaryParams p) {
  using E = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kVec;
  __shared__ float2 cs_all[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* cs = cs_all[warp];
  griddep_wait();
  griddep_launch_dependents();
  const long long task = (long long)blockIdx.x * kWarps + warp;
  if (task >= (long long)p.T * p.parts) return;
  const int t = (int)(task / p.parts), part = (int)(task - (long long)t * p.parts);

  Line line;
  line.per_head = INTER ? p.D / V : p.D / V - p.R / 2 / V;
  line.log_head = 31 - __clz(line.per_head);
  line.inv_head = 1.f / (float)line.per_head;
  line.nq = p.q.nheads * line.per_head;
  line.nk = p.k.nheads * line.per_head;
  line.nv = p.v.nheads * (p.D / V);
  const long long n = line.nq + line.nk + line.nv;
  // shares of whole warps of items
  const int i0 = (int)(n * part / p.parts) & ~31;
  const int i1 = part + 1 == p.parts ? (int)n : (int)(n * (part + 1) / p.parts) & ~31;
  const E* src[3] = {static_cast<const E*>(p.q.src) + t * p.q.src_stride,
                     static_cast<const E*>(p.k.src) + t * p.k.src_stride,
                     static_cast<const E*>(p.v.src) + t * p.v.src_stride};
  Item it[kBatch];
  uint4 a[kBatch], b[kBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + 32 * k;
      if (i >= i1) continue;
      it[k] = item_of<DT, INTER, FIXED>(i, line, p);
      const E* row = it[k].part == 0 ? src[0] : it[k].part == 1 ? src[1] : src[2];
      a[k] = *reinterpret_cast<const uint4*>(row + it[k].at);
      if (!INTER && it[k].mate >= 0) b[k] = *reinterpret_cast<const uint4*>(row + it[k].mate);
    }
  };
  load(i0 + lane);

  // Phases: the top 32 bits as a signed fraction of a half turn.
  const long long pos = p.positions[t];
  for (int i = lane; i < p.R / 2; i += 32) {
    const unsigned long long phase = (unsigned long long)pos * p.steps[i];
    const int top = (int)(unsigned)((phase + 0x80000000ull) >> 32);  // 2^-32 turns
    float s, c;
    sincospif((float)top * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    cs[i] = make_float2(p.factor * c, p.factor * p.sin_sign * s);
  }
  __syncwarp();

  long long slot = -1;  // pool row of this token's K and V
  if (p.key_cache) {
    // Owner sequence: the largest s with cum[s] <= t, 32 candidates at a
    // time; rows at and behind cum[batch] are padding.
    int lo = 0;
    for (int left = p.batch; left > 1;) {
      const int step = (left + 31) / 32, probe = lo + lane * step;
      const unsigned le = __ballot_sync(0xffffffffu, lane * step < left && p.cum[min(probe, p.batch)] <= t);
      const int k = max(__popc(le) - 1, 0);
      lo += k * step;
      left = min(step, left - k * step);
    }
    const int c0 = p.cum[lo], c1 = p.cum[lo + 1], end = p.cum[p.batch];
    const bool note = lane == 0 && part == 0;
    if (t == 0 && part == p.parts - 1) {  // one warp looks over the lengths
      bool bad = p.cum[0] != 0 || end > p.T;
      for (int i = lane; i < p.batch; i += 32) bad |= p.cum[i + 1] < p.cum[i];
      if (bad) atomicOr(p.err, PA_DEVERR_CUM);
    }
    if (t >= end) return;
    if (t < c0 || t >= c1 || c0 < 0) {
      if (note) atomicOr(p.err, PA_DEVERR_CUM);
      return;
    }
    const int past = p.past[lo];
    const long long at = (long long)past + (t - c0);
    if (past < 0) {
      if (note) atomicOr(p.err, PA_DEVERR_PAST);
      return;
    }
    if (at >= (long long)p.MB * p.bs) {
      if (note) atomicOr(p.err, PA_DEVERR_KV_BOUND);
      return;
    }
    const int blk = p.block_table[(size_t)lo * p.MB + at / p.bs];
    if (blk >= 0 && blk < p.NB) slot = (long long)blk * p.bs + at % p.bs;
    else if (blk != -1 && note) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
  }

  E* dst[3] = {static_cast<E*>(p.q.dst) + t * p.q.dst_stride,
               p.key_cache ? static_cast<E*>(p.key_cache) + slot * p.k.nheads * p.D
                           : static_cast<E*>(p.k.dst) + t * p.k.dst_stride,
               p.key_cache ? static_cast<E*>(p.value_cache) + slot * p.v.nheads * p.D : nullptr};
  const bool kv = !p.key_cache || slot >= 0;  // K and V are stored
  constexpr int kTurns = INTER ? V / 2 : V;  // pairs of an item
  float2 w[kTurns];
  auto turns_of = [&](int pair) {
#pragma unroll
    for (int e = 0; e < kTurns; ++e) w[e] = cs[pair + e];
  };
  if constexpr (FIXED) turns_of((lane & (line.per_head - 1)) * kTurns);
  for (int base = i0 + lane;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (base + 32 * k >= i1 || (it[k].part != 0 && !kv)) continue;
      E* row = it[k].part == 0 ? dst[0] : it[k].part == 1 ? dst[1] : dst[2];
      if (it[k].pair >= 0) {
        float x[V];
        unpack<DT>(a[k], x);
        if constexpr (!FIXED) turns_of(it[k].pair);
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 u = w[e / 2];
            const float y1 = x[e] * u.x - x[e + 1] * u.y, y2 = x[e + 1] * u.x + x[e] * u.y;
            x[e] = y1;
            x[e + 1] = y2;
          }
        } else {
          float z[V];
          unpack<DT>(b[k], z);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float y1 = x[e] * w[e].x - z[e] * w[e].y, y2 = z[e] * w[e].x + x[e] * w[e].y;
            x[e] = y1;
            z[e] = y2;
          }
          *reinterpret_cast<uint4*>(row + it[k].mate) = pack<DT>(z);
        }
        a[k] = pack<DT>(x);
      }
      *reinterpret_cast<uint4*>(row + it[k].at) = a[k];
    }
    base += 32 * kBatch;
    if (base - lane >= i1) break;
    load(base);
  }
}

template <int DT, bool INTER>
cudaError_t launch_di(const RotaryParams& p, cudaStream_t s) {
  const unsigned blocks = (unsigned)(((long long)p.T * p.parts + kWarps - 1) / kWarps);
  const int V = Elem<DT>::kVec, per_head = INTER ? p.D / V : p.D / V / 2;
  if (p.R == p.D && per_head <= 32 && (per_head & (per_head - 1)) == 0)
    return launch_pdl(rotary_kernel<DT, INTER, true>, dim3(blocks), kWarps * 32, 0, s, p);
  return launch_pdl(rotary_kernel<DT, INTER, false>, dim3(blocks), kWarps * 32, 0, s, p);
}

template <int DT>
cudaError_t launch_dt(const RotaryParams& p, int interleaved, cudaStream_t s) {
  return interleaved ? launch_di<DT, true>(p, s) : launch_di<DT, false>(p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p0, int dtype, int interleaved, cudaStream_t s) {
  RotaryParams p = p0;
  const int V = dtype == PA_ROTARY_FP32 ? 4 : 8;
  const int per_head = interleaved ? p.D / V : p.D / V - p.R / 2 / V;
  const int items = (p.q.nheads + p.k.nheads) * per_head + p.v.nheads * (p.D / V);
  // A warp's share: one batch of loads (kBatch vectors a lane) while the
  // tokens are few, the whole row once there are enough warps to fill the
  // GPU with loads anyway.
  const int most = std::max(1, (items + 32 * kBatch - 1) / (32 * kBatch));
  const long long want = kWantWarps / std::max(1, p.T) + 1;
  p.parts = (int)std::min<long long>(most, want);
  switch (dtype) {
    case PA_ROTARY_FP16: return launch_dt<PA_ROTARY_FP16>(p, interleaved, s);
    case PA_ROTARY_BF16: return launch_dt<PA_ROTARY_BF16>(p, interleaved, s);
    case PA_ROTARY_FP32: return launch_dt<PA_ROTARY_FP32>(p, interleaved, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
