// Attention for a tree of drafted tokens, the plain way: one warp per
// (packed row, query head), its lanes over the channels, one key at a time
// with the running maximum and sum of the softmax in fp32.
#include "ptx.cuh"
#include "step.h"
#include "tree.h"

namespace pa {
namespace {

constexpr int kWarps = 8;

template <int D, bool BF>
__global__ void __launch_bounds__(kWarps * 32) tree_simple_kernel(const TreeParams p) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  griddep_wait();
  const long long idx = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (idx >= (long long)p.T * p.H) return;
  const int t = (int)(idx / p.H), h = (int)(idx - (long long)t * p.H), k = h / p.G;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cum[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo, c0 = p.cum[b], c1 = p.cum[b + 1], end = p.cum[p.batch];
  const bool note = lane == 0 && h == 0;
  if (t == 0 && h == 0) {
    bool bad = p.cum[0] != 0 || end > p.T;
    for (int i = lane; i < p.batch; i += 32) bad |= p.cum[i + 1] < p.cum[i];
    if (bad) atomicOr(p.err, PA_DEVERR_CUM);
  }
  if (t >= end) return;
  const int past = p.past[b];
  int bits = 0;
  if (t < c0 || t >= c1 || c0 < 0) bits = PA_DEVERR_CUM;
  else if (past < 0) bits = PA_DEVERR_PAST;
  else if (c1 - c0 > p.max_draft) bits = PA_DEVERR_Q_BOUND;
  else if ((long long)past + c1 - c0 > p.max_kv) bits = PA_DEVERR_KV_BOUND;
  if (bits) {
    if (note) atomicOr(p.err, bits);
    return;
  }
  const int n = c1 - c0, j = t - c0;
  const int qpos = p.positions ? p.positions[t] : past + j;
  const int lo_pos = p.window >= 1 ? max(qpos, past) - p.window : -1;  // admitted: position > lo_pos
  float q[kPer], acc[kPer];
  for (int i = 0; i < kPer; ++i) {
    q[i] = elem16_to_float(p.query[((size_t)t * p.H + h) * D + lane * kPer + i], BF);
    acc[i] = 0.f;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  const int first = p.window >= 1 ? max(0, past + 1 - p.window) : 0;
  for (int s = first; s < past + n; ++s) {
    const int blk = p.block_table[(size_t)b * p.MB + (s >> p.log_bs)];
    if (blk < 0 || blk >= p.NB) {
      if (blk != -1 && note) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
      continue;
    }
    int kpos = s;
    if (s >= past) {
      const int i = s - past;
      if (p.mask ? !((p.mask[(size_t)t * p.words + (i >> 5)] >> (i & 31)) & 1) : i > j) continue;
      kpos = p.positions ? p.positions[c0 + i] : s;
    }
    if (p.window >= 1 && kpos <= lo_pos) continue;
    const size_t row = (((size_t)blk << p.log_bs) + (s & (p.bs - 1))) * p.Hk + k;
    float x = 0.f;
    for (int i = 0; i < kPer; ++i) x += q[i] * elem16_to_float(p.key_cache[row * D + lane * kPer + i], BF);
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= p.scale;
    if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
    x += slope * (float)((long long)kpos - qpos);
    const float m_new = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : expf(m - m_new), e = expf(x - m_new);
    l = l * f + e;
    for (int i = 0; i < kPer; ++i)
      acc[i] = acc[i] * f + e * elem16_to_float(p.value_cache[row * D + lane * kPer + i], BF);
    m = m_new;
  }
  if (p.head_sink && m != -INFINITY) l += expf(elem16_to_float(p.head_sink[h], BF) - m);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < kPer; ++i)
    p.out[((size_t)t * p.H + h) * D + lane * kPer + i] = float_to_elem16(acc[i] * inv, BF);
}

}  // namespace

cudaError_t launch_tree_simple(const TreeParams& p, int bf16, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.T * p.H + kWarps - 1) / kWarps);
  if (p.D == 64)
    return bf16 ? launch_pdl(tree_simple_kernel<64, true>, dim3(grid), kWarps * 32, 0, s, p)
                : launch_pdl(tree_simple_kernel<64, false>, dim3(grid), kWarps * 32, 0, s, p);
  return bf16 ? launch_pdl(tree_simple_kernel<128, true>, dim3(grid), kWarps * 32, 0, s, p)
              : launch_pdl(tree_simple_kernel<128, false>, dim3(grid), kWarps * 32, 0, s, p);
}

}  // namespace pa
