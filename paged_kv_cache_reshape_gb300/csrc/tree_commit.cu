// Commit of accepted draft tokens: within each sequence, slot past + i takes
// the K and V rows of slot past + a_i (a_0 < a_1 < ...), in every layer.
//
// In place without a copy: a_i >= i because the path ascends, so a row that
// is overwritten (i) can be the source only of entries up to i.  A thread
// owns one 16-byte column of the rows and walks i upwards, loading a batch
// of sources before it stores them; no other thread touches its column.
//
// Bound by memory (each moved row is read and written once) or, for a few
// rows, by the chain count -> path -> page -> row.  A block serves one
// sequence, checks its path and finds its slots once, and then moves the rows
// of its share of the pools.
//
// Measured (one GB300, 6780 GB/s copied): 128 sequences, up to 12 of 32
// drafts, 80 layers of 8 heads of 128 (390 MB moved) 65 us = 6.0 TB/s; one
// sequence over 32 layers 5.3 to 5.9 us, the host's time to check and launch.
#include <algorithm>

#include "ptx.cuh"
#include "step.h"
#include "tree.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 8;  // rows a thread loads before it stores

__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ long long from[kTreeMaxDraft], to[kTreeMaxDraft];
  __shared__ int n_moves, bad;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x;
  const bool note = blockIdx.y == 0;
  const int past = p.past[b], count = p.count[b];
  if (threadIdx.x == 0) {
    n_moves = 0;
    bad = 0;
  }
  __syncthreads();
  const bool range_ok = past >= 0 && count >= 0 && count <= p.max_accepted;
  const int n = range_ok ? count : 0;
  const int* path = p.accepted + (size_t)b * p.max_accepted;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int a = path[i], before = i > 0 ? path[i - 1] : -1;
    from[i] = -1;
    to[i] = -1;
    // Each entry is looked up only if it can stand at i of an ascending path
    // (a >= i), whatever the others are: slots past + i <= past + a then lie
    // in the sequence's row of the table.
    if (a <= before || a < i || a >= p.max_draft || (long long)past + a >= (long long)p.MB * p.bs) {
      bad = 1;  // (every writer stores the same value)
    } else if (a != i) {
      const int* row = p.block_table + (size_t)b * p.MB;
      const int sb = row[(past + a) / p.bs], db = row[(past + i) / p.bs];
      if (sb >= p.NB || db >= p.NB || sb < -1 || db < -1) {
        if (note) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
      } else if (sb >= 0 && db >= 0) {
        from[i] = (long long)sb * p.bs + (past + a) % p.bs;
        to[i] = (long long)db * p.bs + (past + i) % p.bs;
      }
      if (from[i] >= 0) atomicMax(&n_moves, i + 1);
    }
  }
  __syncthreads();
  const bool ok = range_ok && !bad;
  if (note && threadIdx.x == 0) {
    if (!ok) atomicOr(p.err, past < 0 ? PA_DEVERR_PAST : PA_DEVERR_ACCEPTED);
    if (p.new_past) p.new_past[b] = ok ? past + count : past;
  }
  if (!ok) return;
  const int m = n_moves;  // entries behind the last move need nothing
  if (m == 0) return;
  const int work = p.n_pools * p.row_vecs;
  for (int w = blockIdx.y * kThreads + threadIdx.x; w < work; w += gridDim.y * kThreads) {
    const int pool = w / p.row_vecs, col = w - pool * p.row_vecs;
    uint4* base = static_cast<uint4*>(p.pools[pool]) + col;
    for (int i0 = 0; i0 < m; i0 += kRows) {
      uint4 v[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (i0 + k < m && from[i0 + k] >= 0) v[k] = base[from[i0 + k] * p.row_vecs];
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (i0 + k < m && from[i0 + k] >= 0) base[to[i0 + k] * p.row_vecs] = v[k];
    }
  }
}

}  // namespace

cudaError_t launch_commit(const CommitParams& p, int num_sms, cudaStream_t s) {
  const int shares = std::max(1, (p.n_pools * p.row_vecs + kThreads - 1) / kThreads);
  // Blocks for about two waves of 16 per SM, at most one per 128 columns.
  const int want = std::max(1, (2 * 16 * num_sms + p.batch - 1) / p.batch);
  return launch_pdl(commit_kernel, dim3((unsigned)p.batch, (unsigned)std::min(shares, want)), kThreads, 0, s, p);
}

}  // namespace pa
