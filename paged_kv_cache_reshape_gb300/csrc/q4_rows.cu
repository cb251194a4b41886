// K and V rows to and from pools held in 4 bits.
//
// 32 consecutive channels of a row share a scale s = fp16(a / 7), a their
// largest magnitude, and a channel's code is x / s rounded to nearest even:
// the largest code is 7, so s's own rounding (up to half a step of fp16)
// leaves every value within half a step of s.  Both divisions are IEEE, in
// 32 bits, so the codes are the same bits on every machine.
//
// Bound by memory.  A warp takes 16 packed rows and a share of their K and V
// heads, one head at a time: a row's head is D / 8 lanes of 8 channels, four
// neighbouring lanes a group.  16 rows, because the pool holds a group's
// scales of neighbouring rows side by side: a warp that took one row would
// touch a 32-byte sector for every two bytes of scales.
//
// 52,600 rows of 8 heads of 128, bf16, K and V: written in 73 us (276 MB, 3.8
// TB/s), read in 54 us (5.1 TB/s); with a row to a warp and a division per
// code both took 213 us, now 127.  Instructions issue 63 % of the time, the
// quotients' and the codes' arithmetic, with half the memory's rate used.  A
// decode step's single row is the host's time to check and launch (4.7 us a
// call).
#include <algorithm>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "q4.h"
#include "step.h"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;             // packed rows of a warp
constexpr int kWantWarps = 152 * 32;  // enough to keep the memory busy

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
      f[2 * i] = __low2float(h);
      f[2 * i + 1] = __high2float(h);
    }
  }
}

// The larger of two pairs of non-negative 16-bit values; NaN if one is.
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (BF) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  } else {
    const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

constexpr float kMagic = 12582912.f + 8.f;  // 1.5 2^23 + 8: added to x, leaves 8 + rint(x) in the low bits
constexpr uint32_t kMagicBits = 0x4B400000u;
constexpr float kSnap = 1536.f;              // 1.5 2^10: added and taken off, leaves multiples of 2^-13

// Eight codes by division; apart, since it is rarely run and long.
template <bool BF>
__device__ __noinline__ uint32_t divided(uint4 x, float scale) {
  float f[8];
  unpack8<BF>(x, f);
  uint32_t w = 0;
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const float q = fminf(fmaxf(__fdiv_rn(f[e], scale), -8.f), 7.f);
    w |= (__float_as_uint(q + kMagic) & 15u) << (4 * ((e & 1) * 4 + (e >> 1)));
  }
  return w;
}

// a / 7 rounded to nearest, as an IEEE division gives it for every magnitude
// a of 16 bits whose quotient fp16 tells from 0: the product with 1 / 7, and
// one correction by its remainder, which a fused multiply-add leaves exact
// (Markstein's division).
__device__ __forceinline__ float seventh(float a) {
  const float q = a * (1.f / 7.f);
  return fmaf(fmaf(-7.f, q, a), 1.f / 7.f, q);
}

template <int D, bool BF, bool READ>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 3) q4_rows_kernel(const __grid_constant__ Q4RowsParams p) {
  constexpr int kLanes = D / 8;              // of a row's head
  constexpr int kAtOnce = 32 / kLanes;       // rows that a warp loads in one instruction
  constexpr int kIter = kRows / kAtOnce;
  constexpr int kGroups = D / 32;
  __shared__ __half scales[kWarps][kGroups][kRows];
  const Q4Paging& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const long long task = (long long)blockIdx.x * kWarps + warp;
  const int tiles = (g.T + kRows - 1) / kRows;
  if (task >= (long long)tiles * p.parts) return;
  const int tile = (int)(task / p.parts), part = (int)(task - (long long)tile * p.parts);
  const int h0 = 2 * g.Hk * part / p.parts, h1 = 2 * g.Hk * (part + 1) / p.parts;  // K heads, then V heads

  // Lane i < 16: the slot of packed row 16 tile + i (-1: no such row or
  // page, -2: padding or a row of a bad sequence).
  long long slot = -2;
  {
    const int t = tile * kRows + lane;
    const bool note = part == 0;
    if (task == 0 && bad_cum(g, lane)) atomicOr(g.err, PA_DEVERR_CUM);
    if (lane < kRows && t < g.T && t < g.cum[g.batch]) {
      int lo = 0, hi = g.batch - 1;  // the largest b with cum[b] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.cum[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int c0 = g.cum[lo], c1 = g.cum[lo + 1], past = g.past[lo];
      if (t < c0 || t >= c1 || c0 < 0 || c1 > g.T) {
        if (note) atomicOr(g.err, PA_DEVERR_CUM);
      } else if (past < 0) {
        if (note) atomicOr(g.err, PA_DEVERR_PAST);
      } else if ((long long)past + (c1 - c0) > g.max_kv) {
        if (note) atomicOr(g.err, PA_DEVERR_KV_BOUND);
      } else {
        const int at = past + (t - c0);
        const int blk = g.block_table[(size_t)lo * g.MB + (at >> g.log_bs)];
        slot = blk >= 0 && blk < g.NB ? ((long long)blk << g.log_bs) + (at & (g.bs - 1)) : -1;
        if (slot < 0 && blk != -1 && note) atomicOr(g.err, PA_DEVERR_BLOCK_ID);
      }
    }
  }

  const int c = lane % kLanes, sub = lane / kLanes;  // 8 channels of the head, row of an instruction
  const int j = c >> 2, chunk = c & 3;
  const int run = q4_run_bytes(g.bs, D);
  // Of each row that this lane has a part of: where its word is in head 0's
  // run (negative as the slot is).
  long long at[kIter];
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const long long s = __shfl_sync(0xffffffffu, slot, k * kAtOnce + sub);
    const int r = (int)(s & (g.bs - 1));
    at[k] = s < 0 ? s : (s >> g.log_bs) * g.Hk * run + r * (D / 2) + ((chunk ^ ((r >> 2) & 3)) * kGroups + j) * 4;
  }
  // Scales: lane's pairs of neighbouring rows, of a group each.
  constexpr int kPairs = kGroups * kRows / 2, kPairIter = (kPairs + 31) / 32;

  for (int h = h0; h < h1; ++h) {
    const int v = h >= g.Hk, head = h - v * g.Hk;
    __half* rows = static_cast<__half*>(p.rows[v]) + (size_t)head * D + c * 8;
    uint8_t* runs = p.pool[v] + (size_t)head * run;
    auto word_of = [&](long long at) { return reinterpret_cast<uint32_t*>(runs + at); };
    auto scale_of = [&](long long s, int group) {
      const int r = (int)(s & (g.bs - 1));
      return reinterpret_cast<__half*>(runs + (size_t)(s >> g.log_bs) * g.Hk * run + g.bs * (D / 2)) + group * g.bs + r;
    };
    if constexpr (READ) {
      uint32_t w[kIter];
#pragma unroll
      for (int k = 0; k < kIter; ++k) w[k] = at[k] >= 0 ? *word_of(at[k]) : 0x88888888u;  // (eights: +0)
#pragma unroll
      for (int q = 0; q < kPairIter; ++q) {
        const int x = lane + 32 * q, group = x / (kRows / 2), r2 = x % (kRows / 2) * 2;
        const long long s0 = __shfl_sync(0xffffffffu, slot, r2), s1 = __shfl_sync(0xffffffffu, slot, r2 + 1);
        if (x < kPairs) {
          __half a = __ushort_as_half(0), b = a;  // an unmapped page holds zeros
          if (s0 >= 0) a = *scale_of(s0, group);
          if (s1 >= 0) b = *scale_of(s1, group);
          *reinterpret_cast<__half2*>(&scales[warp][group][r2]) = __halves2half2(a, b);
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kIter; ++k) {
        const int i = k * kAtOnce + sub;
        if (at[k] == -2) continue;
        const float s = __half2float(scales[warp][j][i]);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)((int)(w[k] >> (4 * ((e & 1) * 4 + (e >> 1))) & 15) - 8) * s;
        *reinterpret_cast<uint4*>(rows + (long long)(tile * kRows + i) * p.stride[v]) =
            make_uint4(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]), pack2<BF>(f[4], f[5]), pack2<BF>(f[6], f[7]));
      }
    } else {
      uint4 x[kIter];
#pragma unroll
      for (int k = 0; k < kIter; ++k)
        x[k] = at[k] >= 0 ? *reinterpret_cast<const uint4*>(rows + (long long)(tile * kRows + k * kAtOnce + sub) * p.stride[v])
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kIter; ++k) {
        uint32_t m = max2<BF>(max2<BF>(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu), max2<BF>(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
        m = max2<BF>(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max2<BF>(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max2<BF>(m, m >> 16);
        const uint32_t top = m & 0xffffu;  // bits of the largest magnitude
        const bool finite = top < (BF ? 0x7f80u : 0x7c00u);
        const float a = elem16_to_float(__ushort_as_half((unsigned short)top), BF);
        const __half s = finite ? __float2half_rn(fminf(seventh(a), 65504.f)) : __ushort_as_half((unsigned short)0x7fff);
        const float sf = finite ? __half2float(s) : 0.f;
        // Codes without a division each.  x times about 1 / s is within
        // 2^-18 of x / s.  x and s have 11 bits at most, so x / s is the
        // middle between two whole numbers exactly or at least 2^-13 away
        // from it; rounded to multiples of 2^-13 first (by adding kSnap and
        // taking it off), the product therefore rounds as the quotient does,
        // ties to even included.  Scales so small or large that codes past 7
        // come up are left to a division and a clamp.
        float f[8];
        unpack8<BF>(x[k], f);
        uint32_t w = 0x88888888u;  // zeros
        if (sf >= 6.2e-5f && sf < 65000.f) {
          const float inv = rcp(sf);
          const uint64_t inv2 = f2(inv, inv), magic2 = f2(kMagic, kMagic);
          const uint64_t snap2 = f2(kSnap, kSnap), back2 = f2(-kSnap, -kSnap);
          w = 0;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float r0, r1;
            unf2(add2(add2(add2(mul2(f2(f[e], f[e + 1]), inv2), snap2), back2), magic2), r0, r1);
            // (the magic's own bits leave the sum again below)
            w += __float_as_uint(r0) << (4 * (e >> 1));
            w += __float_as_uint(r1) << (4 * (4 + (e >> 1)));
          }
          w -= kMagicBits * 0x11111111u;
        } else if (sf > 0.f) {
          w = divided<BF>(x[k], sf);
        }
        if (at[k] >= 0) *word_of(at[k]) = w;
        if (chunk == 0) scales[warp][j][k * kAtOnce + sub] = s;
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kPairIter; ++q) {
        const int i = lane + 32 * q, group = i / (kRows / 2), r2 = i % (kRows / 2) * 2;
        const long long s0 = __shfl_sync(0xffffffffu, slot, r2), s1 = __shfl_sync(0xffffffffu, slot, r2 + 1);
        if (i < kPairs) {
          const __half2 both = *reinterpret_cast<const __half2*>(&scales[warp][group][r2]);
          if (s0 >= 0 && s1 == s0 + 1 && !(s0 & 1)) {  // neighbours in a page, at an even row
            *reinterpret_cast<__half2*>(scale_of(s0, group)) = both;
          } else {
            if (s0 >= 0) *scale_of(s0, group) = __low2half(both);
            if (s1 >= 0) *scale_of(s1, group) = __high2half(both);
          }
        }
      }
    }
    __syncwarp();
  }
}

template <int D>
cudaError_t launch_d(const Q4RowsParams& p, bool bf16, bool read, cudaStream_t s) {
  const long long tiles = (p.g.T + kRows - 1) / kRows;
  const dim3 grid((unsigned)((tiles * p.parts + kWarps - 1) / kWarps));
  auto kernel = read ? (bf16 ? q4_rows_kernel<D, true, true> : q4_rows_kernel<D, false, true>)
                     : (bf16 ? q4_rows_kernel<D, true, false> : q4_rows_kernel<D, false, false>);
  return launch_pdl(kernel, grid, kWarps * 32, 0, s, p);
}

}  // namespace

cudaError_t launch_q4_rows(const Q4RowsParams& p0, bool bf16, bool read, cudaStream_t s) {
  Q4RowsParams p = p0;
  // A head to a warp while the rows are few, more once they fill the GPU.
  const long long tiles = (p.g.T + kRows - 1) / kRows;
  p.parts = (int)std::min<long long>(2 * p.g.Hk, kWantWarps / tiles + 1);
  return p.g.D == 64 ? launch_d<64>(p, bf16, read, s) : p.g.D == 128 ? launch_d<128>(p, bf16, read, s)
                                                                     : launch_d<256>(p, bf16, read, s);
}

}  // namespace pa
