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
// through shared memory.  A warp takes one token and a share of its head
// items (an item is one 16-byte vector, or the two of a pair of halves); the
// share shrinks when tokens are few, so that a short draft still fills
// several warps with independent loads.
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

// Where item i of a row starts, its partner vector (half layout), and the
// first pair it turns (-1: copied).
struct Item {
  int at, mate, pair;
};

template <int DT, bool INTER>
__device__ __forceinline__ Item item_of(int i, int per_head, const RotaryParams& p) {
  constexpr int V = Elem<DT>::kVec;
  const int h = i / per_head, c = i - h * per_head;
  Item it;
  if constexpr (INTER) {
    const int ch = c * V;
    const bool rot = ch >= p.off && ch < p.off + p.R;
    it.at = h * p.D + ch;
    it.mate = -1;
    it.pair = rot ? (ch - p.off) / 2 : -1;
  } else {
    const int pairs = p.R / 2 / V;
    if (c < pairs) {
      it.at = h * p.D + p.off + c * V;
      it.mate = it.at + p.R / 2;
      it.pair = c * V;
    } else {
      const int ch = (c - pairs) * V;
      it.at = h * p.D + (ch < p.off ? ch : ch + p.R);
      it.mate = -1;
      it.pair = -1;
    }
  }
  return it;
}

// Rotates (or, with rotate false, copies) items [i0, i1) of one row.
template <int DT, bool INTER>
__device__ __forceinline__ void do_row(const typename Elem<DT>::T* src, typename Elem<DT>::T* dst, int i0, int i1,
                                       int per_head, const RotaryParams& p, const float2* cs, int lane) {
  constexpr int V = Elem<DT>::kVec;
  for (int base = i0 + lane; base < i1; base += 32 * kBatch) {
    Item it[kBatch];
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + 32 * k;
      if (i < i1) {
        it[k] = item_of<DT, INTER>(i, per_head, p);
        a[k] = *reinterpret_cast<const uint4*>(src + it[k].at);
        if (!INTER && it[k].mate >= 0) b[k] = *reinterpret_cast<const uint4*>(src + it[k].mate);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (base + 32 * k >= i1) continue;
      if (it[k].pair >= 0) {
        float x[V];
        unpack<DT>(a[k], x);
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 t = cs[it[k].pair + e / 2];
            const float y1 = x[e] * t.x - x[e + 1] * t.y, y2 = x[e + 1] * t.x + x[e] * t.y;
            x[e] = y1;
            x[e + 1] = y2;
          }
        } else {
          float z[V];
          unpack<DT>(b[k], z);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 t = cs[it[k].pair + e];
            const float y1 = x[e] * t.x - z[e] * t.y, y2 = z[e] * t.x + x[e] * t.y;
            x[e] = y1;
            z[e] = y2;
          }
          *reinterpret_cast<uint4*>(dst + it[k].mate) = pack<DT>(z);
        }
        a[k] = pack<DT>(x);
      }
      *reinterpret_cast<uint4*>(dst + it[k].at) = a[k];
    }
  }
}

template <int DT, bool INTER>
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

  long long slot = -1;  // pool row of this token's K and V
  if (p.key_cache) {
    // Owner sequence: the largest b with cum[b] <= t; rows at and behind
    // cum[batch] are padding.
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cum[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int c0 = p.cum[lo], c1 = p.cum[lo + 1];
    const int end = p.cum[p.batch];
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

  const long long pos = p.positions[t];
  for (int i = lane; i < p.R / 2; i += 32) {
    const unsigned long long phase = (unsigned long long)pos * p.steps[i];
    const int top = (int)(unsigned)((phase + 0x80000000ull) >> 32);  // 2^-32 turns, signed
    float s, c;
    sincospif((float)top * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    cs[i] = make_float2(p.factor * c, p.factor * p.sin_sign * s);
  }
  __syncwarp();

  // The token's items in one line: Q's, K's, then V's plain vectors.
  const int per_head = INTER ? p.D / V : p.D / V - p.R / 2 / V;
  const int nq = p.q.nheads * per_head, nk = p.k.nheads * per_head, nv = p.v.nheads * (p.D / V);
  const long long n = nq + nk + nv;
  const int i0 = (int)(n * part / p.parts), i1 = (int)(n * (part + 1) / p.parts);
  if (i0 < nq)
    do_row<DT, INTER>(static_cast<const E*>(p.q.src) + t * p.q.src_stride,
                      static_cast<E*>(p.q.dst) + t * p.q.dst_stride, i0, min(i1, nq), per_head, p, cs, lane);
  if (p.key_cache && slot < 0) return;
  if (i0 < nq + nk && i1 > nq) {
    E* dst = p.key_cache ? static_cast<E*>(p.key_cache) + slot * p.k.nheads * p.D
                         : static_cast<E*>(p.k.dst) + t * p.k.dst_stride;
    do_row<DT, INTER>(static_cast<const E*>(p.k.src) + t * p.k.src_stride, dst, max(i0 - nq, 0), min(i1 - nq, nk),
                      per_head, p, cs, lane);
  }
  if (i1 > nq + nk) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const E*>(p.v.src) + t * p.v.src_stride);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<E*>(p.value_cache) + slot * p.v.nheads * p.D);
    const int v1 = i1 - nq - nk;
    for (int i = max(i0 - nq - nk, 0) + lane; i < v1; i += 32 * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + 32 * k < v1) v[k] = src[i + 32 * k];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + 32 * k < v1) dst[i + 32 * k] = v[k];
    }
  }
}

template <int DT>
cudaError_t launch_dt(const RotaryParams& p, int interleaved, cudaStream_t s) {
  const long long blocks = ((long long)p.T * p.parts + kWarps - 1) / kWarps;
  if (interleaved) return launch_pdl(rotary_kernel<DT, true>, dim3((unsigned)blocks), kWarps * 32, 0, s, p);
  return launch_pdl(rotary_kernel<DT, false>, dim3((unsigned)blocks), kWarps * 32, 0, s, p);
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
  const long long want = 8192 / std::max(1, p.T) + 1;
  p.parts = (int)std::min<long long>(most, want);
  switch (dtype) {
    case PA_ROTARY_FP16: return launch_dt<PA_ROTARY_FP16>(p, interleaved, s);
    case PA_ROTARY_BF16: return launch_dt<PA_ROTARY_BF16>(p, interleaved, s);
    case PA_ROTARY_FP32: return launch_dt<PA_ROTARY_FP32>(p, interleaved, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
