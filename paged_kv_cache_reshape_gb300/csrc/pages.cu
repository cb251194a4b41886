// Pages of a cache: copies, forks of sequences, growth and release, and
// compaction, without the host reading a length.
//
// Every call runs a plan (one block: who needs a page, which pages are free,
// what moves where) and then an apply (all SMs: the tables, the reference
// counts and the pages' bytes in every pool).  A page is free when nothing
// refers to it; fresh pages are the lowest free ones, handed to the rows in
// their order, so that a call's result does not depend on how its threads
// run.  Pages that a call releases are free from the next call on.
//
// Bound by memory: each moved page is read and written once in each pool.
// Compaction of 32 sequences in 32 layers' K and V pools (1.08 GB moved): 174
// us, 6.2 TB/s, 92 % of the copy rate.  96 beams forked in 32 layers, then each
// grown by its next token (193 MB): 49 us; the plans, one block's chain of
// scans, are 6 and 8 of them, the pages' copies 29.
// Plan and apply in one launch, the blocks waiting for the first, took 60 us.
#include <algorithm>
#include <climits>

#include "pages.h"
#include "ptx.cuh"
#include "step.h"

namespace pa {
namespace {

constexpr int kPlan = 1024;
constexpr int kApply = 256;

// Exclusive sum over the block's threads of small counts; *total their sum.
// Every thread calls it; shared: kPlan / 32 + 1 words.
__device__ __forceinline__ int block_scan(int v, int* shared, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the words may still be read from the scan before
  if (lane == 31) shared[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = shared[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    shared[lane] = s;
  }
  __syncthreads();
  *total = shared[kPlan / 32 - 1];
  return x - v + (warp ? shared[warp - 1] : 0);
}

// Which of four pages from `at` on have no reference, as bits.
__device__ __forceinline__ int free_of(const int* ref, int NB, int at) {
  int bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i < NB && ref[at + i] == 0) bits |= 1 << i;
  return bits;
}

// The lowest `want` pages with no reference into list; returns how many
// there are (at most want).  head: free_of the first 4 kPlan pages, asked
// for while there was something else to wait for.
__device__ int find_free(const int* ref, int NB, int want, int* list, int* shared, int head) {
  int got = 0;
  for (int base = 0; base < NB && got < want; base += 4 * kPlan) {
    const int at = base + 4 * threadIdx.x, bits = base ? free_of(ref, NB, at) : head;
    int total;
    int rank = got + block_scan(__popc(bits), shared, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (bits >> i & 1) {
        if (rank < want) list[rank] = at + i;
        ++rank;
      }
    }
    got = min(want, got + total);
  }
  __syncthreads();
  return got;
}

__device__ __forceinline__ int pages_of(int length, int bs) { return (int)(((long long)length + bs - 1) / bs); }

// An entry of a table as a page, -1 where there is none.
__device__ __forceinline__ int page_at(const int* entry, int NB, int* err) {
  const int x = *entry;
  if (x >= 0 && x < NB) return x;
  if (x != -1) atomicOr(err, PA_DEVERR_BLOCK_ID);
  return -1;
}

__device__ void plan_copy(const PagesParams& p, int* shared) {
  const int n = p.n_pairs;
  auto inside = [&](int x) { return x >= 0 && x < p.NB; };
  for (int i = threadIdx.x; i < n; i += kPlan) {
    if (inside(p.src[i])) p.w.place[p.src[i]] = 0;
    if (inside(p.dst[i])) p.w.place[p.dst[i]] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (inside(p.src[i]) && inside(p.dst[i])) atomicAdd(&p.w.place[p.dst[i]], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int s = p.src[i], d = p.dst[i];
    const bool out = s == -1 || d == -1;
    const bool ok = inside(s) && inside(d) && p.w.place[d] == 1 && p.w.place[s] == 0;
    p.w.moves[i] = ok ? make_int2(s, d) : make_int2(-1, -1);
    if (!ok && !out) atomicOr(p.err, inside(s) && inside(d) ? PA_DEVERR_PAGES : PA_DEVERR_BLOCK_ID);
  }
  if (threadIdx.x == 0) *p.w.n_moves = n;
}

__device__ void plan_fork(const PagesParams& p, int* shared) {
  auto parent_of = [&](int i, bool note) {
    const int a = p.parent[i];
    if (a >= -1 && a < p.rows_in) return a;
    if (note) atomicOr(p.err, PA_DEVERR_PAGES);
    return -1;
  };
  auto length_of = [&](int a, bool note) {
    const int x = a < 0 ? 0 : p.lengths[a];
    if (x >= 0 && x <= (long long)p.MB * p.bs) return x;
    if (note) atomicOr(p.err, x < 0 ? PA_DEVERR_PAST : PA_DEVERR_KV_BOUND);
    return -1;
  };
  const int head = free_of(p.ref, p.NB, 4 * threadIdx.x);
  for (int r = threadIdx.x; r < p.rows_in; r += kPlan) p.w.first[r] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < p.rows; i += kPlan) {
    const int a = parent_of(i, true);
    if (a >= 0) atomicMin(&p.w.first[a], i);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < p.rows; base += kPlan) {
    const int i = base + threadIdx.x;
    bool need = false;
    if (i < p.rows) {
      const int a = parent_of(i, false), len = length_of(a, true);
      need = a >= 0 && len > 0 && len % p.bs && p.w.first[a] != i &&
             page_at(p.table + (size_t)a * p.MB + len / p.bs, p.NB, p.err) >= 0;
    }
    int total;
    const int rank = want + block_scan(need, shared, &total);
    if (i < p.rows) p.w.fresh[i] = need ? rank : -1;
    want += total;
  }
  const int got = find_free(p.ref, p.NB, min(want, p.NB), p.w.free_list, shared, head);
  for (int i = threadIdx.x; i < p.rows; i += kPlan) {
    const int a = parent_of(i, false), len = max(length_of(a, false), 0), rank = p.w.fresh[i];
    bool ok = true;
    if (rank >= 0) {
      ok = rank < got;
      p.w.fresh[i] = ok ? p.w.free_list[rank] : -1;
      if (ok) p.w.moves[rank] = make_int2(p.table[(size_t)a * p.MB + len / p.bs], p.w.fresh[i]);
      else atomicOr(p.err, PA_DEVERR_PAGES);
    }
    p.w.entries[i] = ok ? pages_of(len, p.bs) : 0;
    p.lengths_out[i] = ok ? len : 0;
  }
  if (threadIdx.x == 0) *p.w.n_moves = got;
}

// A row's lengths before and after a resize; false where they are no lengths.
__device__ __forceinline__ bool resized(const PagesParams& p, int r, int* was, int* now) {
  const long long a = p.lengths[r], b = a + p.delta[r], most = (long long)p.MB * p.bs;
  *was = (int)a;
  *now = (int)b;
  return a >= 0 && a <= most && b >= 0 && b <= most;
}

// Whether a growing row's entry c, which new positions fall into, has to
// become a fresh page: it has none, or one that other rows refer to as well.
// (An entry that holds positions below `was` too and has no page stays so.)
__device__ __forceinline__ bool wants_page(const PagesParams& p, const int* ref, const int* entry, int c, int was) {
  const int page = page_at(entry, p.NB, p.err);
  return page >= 0 ? ref[page] > 1 : (long long)c * p.bs >= was;
}

// The shared page whose bytes a growing row takes along into a fresh one, or
// -1: it holds positions on both sides of `was`.
__device__ __forceinline__ int shared_page(const PagesParams& p, int r, int was, int now) {
  if (now <= was || was % p.bs == 0) return -1;
  const int page = page_at(p.table + (size_t)r * p.MB + was / p.bs, p.NB, p.err);
  return page >= 0 && p.ref[page] > 1 ? page : -1;
}

__device__ void plan_resize(const PagesParams& p, int* shared) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = free_of(p.ref, p.NB, 4 * threadIdx.x);
  // Pages that each row needs: a thread to a row, and a warp to rows that
  // grow by more than a few pages (a prompt; one after the other they would
  // wait for the table's every entry).
  constexpr int kFew = 4;
  for (int r = threadIdx.x; r < p.rows; r += kPlan) {
    int was, now, need = -1;
    if (!resized(p, r, &was, &now)) {
      atomicOr(p.err, was < 0 ? PA_DEVERR_PAST : PA_DEVERR_KV_BOUND);
    } else if (pages_of(now, p.bs) - pages_of(was, p.bs) <= kFew) {
      need = 0;
      for (int c = was / p.bs; now > was && c < pages_of(now, p.bs); ++c)
        need += wants_page(p, p.ref, p.table + (size_t)r * p.MB + c, c, was);
      need = min(need, p.NB + 1);  // (more than there are is too many)
    }
    p.w.entries[r] = need;
  }
  __syncthreads();
  for (int r = warp; r < p.rows; r += kPlan / 32) {
    int was, now, need = 0;
    if (!resized(p, r, &was, &now) || pages_of(now, p.bs) - pages_of(was, p.bs) <= kFew) continue;
    for (int c = was / p.bs + lane; c < pages_of(now, p.bs); c += 32)
      need += wants_page(p, p.ref, p.table + (size_t)r * p.MB + c, c, was);
    need = __reduce_add_sync(0xffffffffu, need);
    if (lane == 0) p.w.entries[r] = min(need, p.NB + 1);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < p.rows; base += kPlan) {
    const int r = base + threadIdx.x, need = r < p.rows ? max(p.w.entries[r], 0) : 0;
    int total;
    const int start = block_scan(need, shared, &total);
    if (r < p.rows) p.w.fresh[r] = (int)min((long long)want + start, (long long)INT_MAX);
    want = (int)min((long long)want + total, (long long)INT_MAX / 2);
  }
  const int got = find_free(p.ref, p.NB, min(want, p.NB), p.w.free_list, shared, head);
  // Rows whose pages are all there are served, entries in their order; the
  // page that is copied is the first of them.
  int moved = 0;
  for (int base = 0; base < p.rows; base += kPlan) {
    const int r = base + threadIdx.x;
    int from = -1, at = 0;
    if (r < p.rows) {
      int was = 0, now = 0;
      const int need = p.w.entries[r];
      bool ok = need >= 0;
      resized(p, r, &was, &now);
      if (ok && need > 0 && (long long)p.w.fresh[r] + need > got) {
        ok = false;
        atomicOr(p.err, PA_DEVERR_PAGES);
      }
      if (!ok) p.w.entries[r] = -1;
      else if (need > 0) from = shared_page(p, r, was, now), at = p.w.fresh[r];
      p.lengths_out[r] = ok ? now : was;
    }
    int total;
    const int rank = moved + block_scan(from >= 0, shared, &total);
    if (from >= 0) p.w.moves[rank] = make_int2(from, p.w.free_list[at]);
    moved += total;
  }
  if (threadIdx.x == 0) *p.w.n_moves = moved;
}

__device__ void plan_compact(const PagesParams& p, int* shared) {
  int live = 0;
  for (int base = 0; base < p.NB; base += 4 * kPlan) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = base + i * kPlan + threadIdx.x;
      n += at < p.NB && p.ref[at] != 0;
    }
    live += n;
  }
  int total;
  block_scan(live, shared, &total);
  live = total;
  const int moves = find_free(p.ref, live, live, p.w.free_list, shared, free_of(p.ref, live, 4 * threadIdx.x));  // the holes below `live`
  int done = 0;
  for (int base = 0; base < p.NB; base += kPlan) {
    const int at = base + threadIdx.x;
    const bool moved = at >= live && at < p.NB && p.ref[at] != 0;
    if (base + kPlan <= live) {
      p.w.place[at] = at;
      continue;
    }
    const int rank = done + block_scan(moved, shared, &total);
    if (moved) p.w.moves[rank] = make_int2(at, p.w.free_list[rank]);
    if (at < p.NB) p.w.place[at] = moved ? p.w.free_list[rank] : at;
    done += total;
  }
  if (threadIdx.x == 0) {
    *p.w.n_moves = moves;
    *p.live = live;
  }
}

template <PageOp OP>
__global__ void __launch_bounds__(kPlan) plan_kernel(const __grid_constant__ PagesParams p) {
  __shared__ int shared[kPlan / 32 + 1];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x > 0) {  // the other blocks carry the counts over, or keep them as they were
    int* to = OP == kPageResize ? p.w.place : p.ref_out;
    for (int i = (blockIdx.x - 1) * kPlan + threadIdx.x; i < p.NB; i += (gridDim.x - 1) * kPlan) to[i] = p.ref[i];
    return;
  }
  if constexpr (OP == kPageCopy) plan_copy(p, shared);
  if constexpr (OP == kPageFork) plan_fork(p, shared);
  if constexpr (OP == kPageResize) plan_resize(p, shared);
  if constexpr (OP == kPageCompact) plan_compact(p, shared);
}

// The new rows of a fork.  A row's first child takes over its references, so
// only other children add some and only rows without one lose theirs.
__device__ void apply_fork(const PagesParams& p, long long i, long long step) {
  for (long long x = i; x < (long long)p.rows * p.MB; x += step) {
    const int r = (int)(x / p.MB), c = (int)(x - (long long)r * p.MB);
    int page = -1;
    const int n = p.w.entries[r];
    if (c < n) {
      const int a = p.parent[r];
      page = page_at(p.table + (size_t)a * p.MB + c, p.NB, p.err);
      if (c == n - 1 && p.w.fresh[r] >= 0) page = p.w.fresh[r];
      if (page >= 0 && p.w.first[a] != r) atomicAdd(&p.ref_out[page], 1);
    }
    p.table_out[x] = page;
  }
  for (long long x = i; x < (long long)p.rows_in * p.MB; x += step) {
    const int r = (int)(x / p.MB), c = (int)(x - (long long)r * p.MB);
    const int child = p.w.first[r];
    if (child != INT_MAX && c < p.w.entries[child]) continue;
    const int page = page_at(p.table + x, p.NB, p.err);
    if (page >= 0) atomicAdd(&p.ref_out[page], -1);
  }
}

__device__ void apply_resize(const PagesParams& p, long long warp, long long warps, int lane) {
  for (long long r = warp; r < p.rows; r += warps) {
    if (p.w.entries[r] < 0) continue;
    int* row = p.table_out + (size_t)r * p.MB;
    const int now = p.lengths_out[r];
    const int was = (int)((long long)now - p.delta[r]);
    int at = p.w.fresh[r];
    // As planned: the counts are those of before the call (place), which this
    // launch changes.
    const int end = p.w.entries[r] > 0 ? pages_of(now, p.bs) : 0;
    for (int c0 = was / p.bs; c0 < end; c0 += 32) {
      const int c = c0 + lane;
      const bool takes = c < end && wants_page(p, p.w.place, row + c, c, was);
      const unsigned takers = __ballot_sync(0xffffffffu, takes);
      if (takes) {
        const int old = row[c], page = p.w.free_list[at + __popc(takers & ((1u << lane) - 1))];
        if (old >= 0 && old < p.NB) atomicAdd(&p.ref_out[old], -1);
        row[c] = page;
        p.ref_out[page] = 1;
      }
      at += __popc(takers);
    }
    for (int c = pages_of(now, p.bs) + lane; c < p.MB; c += 32) {
      const int page = page_at(row + c, p.NB, p.err);
      if (page >= 0) atomicAdd(&p.ref_out[page], -1);
      row[c] = -1;
    }
  }
}

__device__ void apply_compact(const PagesParams& p, long long i, long long step) {
  for (long long x = i; x < (long long)p.rows * p.MB; x += step) {
    const int page = page_at(p.table + x, p.NB, p.err);
    p.table_out[x] = page >= 0 ? p.w.place[page] : -1;
  }
  for (long long m = i; m < *p.w.n_moves; m += step) {
    const int2 mv = p.w.moves[m];
    p.ref_out[mv.y] = p.ref[mv.x];
    p.ref_out[mv.x] = 0;
  }
}

constexpr int kVecs = 4;                      // 16-byte vectors a thread holds
constexpr int kSegment = kApply * kVecs;      // vectors of a segment

template <PageOp OP>
__global__ void __launch_bounds__(kApply) apply_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PageCopyParams c) {
  griddep_wait();
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * kApply + threadIdx.x, step = (long long)gridDim.x * kApply;
  if (c.with_tables) {
    if constexpr (OP == kPageFork) apply_fork(p, i, step);
    if constexpr (OP == kPageResize) apply_resize(p, i >> 5, step >> 5, threadIdx.x & 31);
    if constexpr (OP == kPageCompact) apply_compact(p, i, step);
  }
  const long long segments = (c.page_vecs + kSegment - 1) / kSegment;
  const long long work = (long long)*p.w.n_moves * c.n_pools * segments;
  for (long long x = blockIdx.x; x < work; x += gridDim.x) {
    const long long m = x / (c.n_pools * segments), y = x - m * (c.n_pools * segments);
    const int pool = (int)(y / segments);
    const long long v0 = (y - pool * segments) * kSegment + threadIdx.x;
    const int2 mv = p.w.moves[m];
    if (mv.x < 0) continue;
    uint4* base = static_cast<uint4*>(c.pools[pool]);
    const uint4* from = base + mv.x * c.page_vecs;
    uint4* to = base + mv.y * c.page_vecs;
    uint4 v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (v0 + k * kApply < c.page_vecs) v[k] = from[v0 + k * kApply];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (v0 + k * kApply < c.page_vecs) to[v0 + k * kApply] = v[k];
  }
}

}  // namespace

cudaError_t launch_page_plan(PageOp op, const PagesParams& p, cudaStream_t s) {
  const bool carry = op == kPageResize || (op != kPageCopy && p.ref_out != p.ref);
  const dim3 grid(1 + (carry ? std::min(64, (p.NB + kPlan - 1) / kPlan) : 0));
  switch (op) {
    case kPageCopy: return launch_pdl(plan_kernel<kPageCopy>, grid, kPlan, 0, s, p);
    case kPageFork: return launch_pdl(plan_kernel<kPageFork>, grid, kPlan, 0, s, p);
    case kPageResize: return launch_pdl(plan_kernel<kPageResize>, grid, kPlan, 0, s, p);
    default: return launch_pdl(plan_kernel<kPageCompact>, grid, kPlan, 0, s, p);
  }
}

cudaError_t launch_page_apply(PageOp op, const PagesParams& p, const PageCopyParams& c, int num_sms, cudaStream_t s) {
  const dim3 grid(num_sms * 8);
  switch (op) {
    case kPageCopy: return launch_pdl(apply_kernel<kPageCopy>, grid, kApply, 0, s, p, c);
    case kPageFork: return launch_pdl(apply_kernel<kPageFork>, grid, kApply, 0, s, p, c);
    case kPageResize: return launch_pdl(apply_kernel<kPageResize>, grid, kApply, 0, s, p, c);
    default: return launch_pdl(apply_kernel<kPageCompact>, grid, kApply, 0, s, p, c);
  }
}

}  // namespace pa
