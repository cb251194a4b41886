// Attention for a tree of drafted tokens over the paged cache.
//
// Rows are (draft token, query head of the kv head's group); every row of a
// sequence attends to the same context, so its K and V are read once for up
// to 256 rows.  One pass over the keys with the running maximum m and sum l
// of the softmax:
//   S = Q K^T;  x = S scale (softcap, distance bias), -inf where masked
//   m' = max(m, max x);  P = exp(x - m');  l = l exp(m - m') + sum P;  O = O exp(m - m') + P V
// Partial results over ranges of keys join by out = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s.
//
// Work: a unit is a sequence, a kv head and up to two 128-row tiles; its
// length is its number of 128-key tiles.  All units in a line are cut into
// equal ranges, one per CTA (one CTA per SM), whatever unit borders they
// cross: every SM streams the same number of key tiles, and at most one unit
// border per range is a cut, whose two or more partial results a second small
// kernel joins.  Every CTA finds its range from the lengths by itself (one
// read of the lengths, a block scan), so the step needs no planning launch.
//
// A unit of two row tiles runs them as two streams over the same key tiles;
// a unit of one row tile runs its even and odd key tiles as the two streams
// and joins them at its end, so that either way one stream's softmax overlaps
// the other's tensor work.  Per stream: S and O in tensor memory (S = M 128 x
// N 128 columns, O = head_size columns), P over S as 16-bit pairs, read from
// there by the P V product.
//
// Masks: an interior tile (context only) needs none.  A tile that holds
// draft tokens, a window's edge or an unmapped page builds one 128-bit mask
// per row.  P is zero at masked keys, and 0 * inf would still be NaN in the
// P V product, so V rows past the sequence are zeroed in shared memory, and
// non-finite values in draft rows (which only some rows admit) are taken out
// there and added to the rows that do admit them when O leaves tensor memory.
//
// Roles (384 threads): warpgroups 0 and 1, softmax and epilogue of the two
// streams (thread = row = TMEM lane); warp 8 K/V producer (TMA, a ring of
// slots in the order K0 V0 K1 V1 ...), warp 9 TMEM owner and MMA issuer, warp
// 10 walks the CTA's range, publishes segments and loads Q.
#include "f32x2.cuh"
#include "ptx.cuh"
#include "step.h"
#include "tree.h"

namespace pa {
namespace {

constexpr int kThreads = 12 * 32;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kFetchWarp = 10;
// Registers per thread after the split (launch: 168 each).
constexpr int kRegSoftmax = 208, kRegControl = 80;
static_assert(2 * kRegSoftmax + kRegControl <= 3 * 168, "register split");
constexpr int kKeys = 128;   // keys per K/V tile
constexpr int kRows = 128;   // rows per row tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyRescale = 8.f;  // log2 of the largest P value tolerated before rescaling
constexpr int kSmemLimit = 227 * 1024;
constexpr int kCtrlBytes = 3072;
constexpr int kInfoRing = 4;  // segments published ahead of their use
// Page masks of the K/V tiles in flight: the producer cannot be a whole ring
// ahead of a stream (a slot is reused only after MMAs that follow the softmax
// of all older tiles but the last few).
constexpr int kMaskRing = 8;

template <int D>
struct TreeCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kQTileBytes = kRows * D * 2;  // [chunk][row][128 B]
  static constexpr int kSlotBytes = kKeys * D * 2;   // one K or V tile [chunk][key][128 B]
  static constexpr int kSlotsFit = (kSmemLimit - kCtrlBytes - 2 * kQTileBytes) / kSlotBytes;
  static constexpr int kSlots = kSlotsFit > 8 ? 8 : kSlotsFit;
  static __host__ __device__ constexpr int s_col(int X) { return X * kKeys; }
  static __host__ __device__ constexpr int o_col(int X) { return 2 * kKeys + X * D; }
  static constexpr int kTmemCols = 512;
  static constexpr int kDataBytes = 2 * kQTileBytes + kSlots * kSlotBytes;
  static constexpr int kSmemBytes = kDataBytes + kCtrlBytes;
};

// One range of a unit's key tiles.
struct Segment {
  int live;    // 0: no more work
  int b, k;    // sequence, kv head
  int t0;      // packed row of the unit's first token
  int ntok;    // the unit's tokens
  int two;     // 1: two row tiles (streams are rows), 0: one (streams are even and odd key tiles)
  int seq_t0;  // packed row of the sequence's first draft token
  int n;       // the sequence's draft tokens
  int past;
  int key0;    // position of the first key of the segment's first tile
  int nt;      // key tiles
  int slot;    // partial slot; -1: the whole unit, stored to the output
  int pad[4];
};

struct Ctrl {
  Segment seg[kInfoRing];
  uint32_t kv_mask[kMaskRing];    // per K/V tile (tile number mod ring): its pages that are unmapped
  uint32_t bad[8][kTreeMaxWords];  // per softmax warp: draft tokens of the segment with non-finite V
  float2 ml[2][kRows];            // per stream: running maximum and sum of the segment
  uint64_t mask_full[kMaskRing];
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t info_full[kInfoRing], info_empty[kInfoRing];
  uint64_t xchg_full, xchg_done;
  uint64_t drain;
  long long scan[kThreads / 32];
  long long start_off;  // this CTA's first key tile, within sequence start_b
  int start_b;
  uint32_t tmem_base;
  int abort;
};

// What the schedule needs of a sequence.
struct SeqWork {
  int past, n, t0;
  int lo;        // first key walked (a multiple of 128)
  int nt;        // key tiles of each unit
  int pairs;     // units per kv head
  long long len; // key tiles of all units
};

__device__ __forceinline__ SeqWork seq_work(const TreeParams& p, int b, int& bits) {
  SeqWork s;
  s.t0 = p.cum[b];
  const int t1 = p.cum[b + 1];
  s.past = p.past[b];
  s.n = t1 - s.t0;
  s.len = 0;
  s.nt = s.pairs = s.lo = 0;
  if (s.t0 < 0 || t1 < s.t0 || t1 > p.T || (b == 0 && s.t0 != 0)) {
    bits |= PA_DEVERR_CUM;
  } else if (s.past < 0) {
    bits |= PA_DEVERR_PAST;
  } else if (s.n > p.max_draft) {
    bits |= PA_DEVERR_Q_BOUND;
  } else if ((long long)s.past + s.n > p.max_kv) {
    bits |= PA_DEVERR_KV_BOUND;
  } else if (s.n > 0) {
    s.lo = p.window >= 1 ? (max(0, s.past + 1 - p.window) & ~(kKeys - 1)) : 0;
    s.nt = (s.past + s.n - s.lo + kKeys - 1) / kKeys;
    s.pairs = (s.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    s.len = (long long)s.nt * s.pairs * p.Hk;
  }
  return s;
}

// Draft token i of the sequence admitted by the row of draft token j.
__device__ __forceinline__ bool mask_bit(const TreeParams& p, int t, int j, int i) {
  return p.mask ? (p.mask[(size_t)t * p.words + (i >> 5)] >> (i & 31)) & 1 : i <= j;
}

// Bits [a, b) of a 32-bit word.
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = min(max(a, 0), 32);
  b = min(max(b, 0), 32);
  const uint32_t upto_b = b == 32 ? 0xffffffffu : (1u << b) - 1u;
  const uint32_t upto_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
  return upto_b & ~upto_a;
}

template <bool BF>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
  return BF ? (h & 0x7f80u) == 0x7f80u : (h & 0x7c00u) == 0x7c00u;
}

// GEN: softcap, distance bias or a window (checked at run time); without it
// the scores need one multiplication.
template <int D, bool BF, bool GEN>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  constexpr int S = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_s = smem;                       // [tile A, tile B]
  uint8_t* kv_s = q_s + 2 * C::kQTileBytes;  // [slot]: K_i is load 2i, V_i load 2i+1
  Ctrl* ctl = reinterpret_cast<Ctrl*>(smem + C::kDataBytes);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->o_done[i], 1);
      mbar_init(&ctl->o_free[i], 8);
    }
    for (int i = 0; i < kInfoRing; ++i) {
      mbar_init(&ctl->info_full[i], 1);
      mbar_init(&ctl->info_empty[i], 1 + 8 + 1);  // MMA, softmax and K/V producer warps
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ctl->mask_full[i], 1);
    mbar_init(&ctl->xchg_full, 8);
    mbar_init(&ctl->xchg_done, 8);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ctl->start_b = -1;
    fence_mbar_init();
  }
  if (threadIdx.x < 8 * kTreeMaxWords) ctl->bad[0][threadIdx.x] = 0;
  if (warp == kFetchWarp && lane == 0) prefetch_tmap(&tm_q);
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }

  griddep_wait();  // lengths, queries and pools may come from the previous kernel
  griddep_launch_dependents();

  // The line of all units: its length, and where this CTA's range starts.
  int bits = 0;
  long long total = 0;
  SeqWork mine{};
  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    const SeqWork s = seq_work(p, b, bits);
    if (b == (int)threadIdx.x) mine = s;
    total += s.len;
  }
  if (bits && blockIdx.x == 0) atomicOr(p.err, bits);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) ctl->scan[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += ctl->scan[w];
  const long long active = min((long long)gridDim.x, (total + p.min_tiles - 1) / p.min_tiles);
  if ((smem_u32(smem) & 1023) != 0) {  // the swizzled operands need it; never seen
    if (threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_TIMEOUT);
    if (threadIdx.x == 0) p.cuts[blockIdx.x].rows = 0;
    return;
  }
  if (blockIdx.x >= active) {
    if (threadIdx.x == 0) p.cuts[blockIdx.x].rows = 0;
    return;
  }
  const long long r_begin = total * blockIdx.x / active, r_end = total * (blockIdx.x + 1) / active;
  long long before = 0;  // length of the sequences of earlier rounds
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int ignored = 0;
    long long len = 0;
    if (b < p.batch) len = b0 == 0 ? mine.len : seq_work(p, b, ignored).len;
    long long incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) ctl->scan[warp] = incl;
    __syncthreads();
    long long first = before + incl - len;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) first += ctl->scan[w];
      before += ctl->scan[w];
    }
    if (len > 0 && first <= r_begin && r_begin < first + len) {
      ctl->start_b = b;
      ctl->start_off = r_begin - first;
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int log_r = p.log_page_rows;  // log2(min(block_size, 128))
  const int pages = kKeys >> log_r;

  // Register split: each warpgroup resizes at the top of its own branch
  // (the allocator budgets a branch from the setmaxnreg that dominates it).
  if (warp >= kProducerWarp) {
    regs_dec<kRegControl>();
    if (warp == kFetchWarp) {
      // ---------------------------------------------------------- fetcher
      // Walks the range, publishes its segments and loads their Q tiles once
      // the previous segment's S products are done.
      const uint32_t q_bytes = C::kChunks * p.G * p.tile_tokens * 128;
      int b = ctl->start_b;
      long long off = ctl->start_off, r = r_begin;
      uint32_t q_loads = 0;
      Cut cut{};  // the unit that starts in this range and goes on behind it
      int ignored = 0;
      SeqWork s = seq_work(p, b, ignored);
      for (uint32_t tt = 0;; ++tt) {
        Segment f{};
        if (r < r_end) {
          while (off >= s.len) {  // next sequence with work (one exists: r < total)
            off = 0;
            s = seq_work(p, ++b, ignored);
          }
          const int u = (int)(off / s.nt), tile0 = (int)(off - (long long)u * s.nt);
          const int pair = u % s.pairs;
          f.live = 1;
          f.b = b;
          f.k = u / s.pairs;
          f.t0 = s.t0 + pair * 2 * p.tile_tokens;
          f.ntok = min(2 * p.tile_tokens, s.n - pair * 2 * p.tile_tokens);
          f.two = f.ntok > p.tile_tokens;
          f.seq_t0 = s.t0;
          f.n = s.n;
          f.past = s.past;
          f.key0 = s.lo + tile0 * kKeys;
          f.nt = (int)min((long long)(s.nt - tile0), r_end - r);
          f.slot = f.nt == s.nt ? -1 : 2 * (int)blockIdx.x + (r == r_begin ? 0 : 1);
          if (tile0 == 0 && f.nt < s.nt) {
            // the CTA that holds the unit's last tile: the largest c with total * c / active <= last
            const long long last = r + s.nt - 1;
            cut.rows = f.two ? kRows + (f.ntok - p.tile_tokens) * p.G : f.ntok * p.G;
            cut.slot0 = f.slot;
            cut.more = (int)(((last + 1) * active - 1) / total) - (int)blockIdx.x;
            cut.t0 = f.t0;
            cut.ntok = f.ntok;
            cut.k = f.k;
          }
          off += f.nt;
          r += f.nt;
        }
        const int slot = tt % kInfoRing;
        bool ok = true;
        if (lane == 0) {
          if (!wait_or_abort(&ctl->info_empty[slot], ((tt / kInfoRing) & 1) ^ 1, abort, p.err, p.err_site, kSiteTree | 1)) {
            ok = false;
          } else {
            ctl->seg[slot] = f;
            mbar_arrive(&ctl->info_full[slot]);
            if (f.live) {
              if (!wait_or_abort(&ctl->q_empty, (tt & 1) ^ 1, abort, p.err, p.err_site, kSiteTree | 2)) {
                ok = false;
              } else {
                mbar_arrive_expect_tx(&ctl->q_full, (f.two ? 2 : 1) * q_bytes);
                for (int X = 0; X < (f.two ? 2 : 1); ++X)
                  for (int c = 0; c < C::kChunks; ++c)
                    tma_load_3d(q_s + X * C::kQTileBytes + c * (kRows * 128), &tm_q, c * 64, f.k * p.G,
                                f.t0 + X * p.tile_tokens, &ctl->q_full);
                ++q_loads;
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok || !f.live) break;
      }
      if (lane == 0) {
        p.cuts[blockIdx.x] = cut;
        if (*abort && q_loads > 0) {
          // Gave up: let the copies already issued land before the CTA exits.
          for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&ctl->q_full, (q_loads - 1) & 1); ++i) {
          }
        }
      }
    } else if (warp == kProducerWarp) {
      // ----------------------------------------------------- K/V producer
      uint32_t n_loads = 0;  // K/V slot loads issued so far
      bool ok = true;
      // One K or V tile into the next ring slot: lane l copies page
      // l / chunks, 64-column chunk l % chunks (a box of {64, 1, page rows}).
      auto load_tile = [&](const CUtensorMap* tm, int k, int rc, bool is_v, uint32_t mask) -> bool {
        const int slot = n_loads % S;
        if (lane == 0) {
          if (!wait_or_abort(&ctl->empty[slot], ((n_loads / S) & 1) ^ 1, abort, p.err, p.err_site, kSiteTree | 3)) {
            ok = false;
          } else {
            if (!is_v) {
              ctl->kv_mask[(n_loads >> 1) % kMaskRing] = mask;
              mbar_arrive(&ctl->mask_full[(n_loads >> 1) % kMaskRing]);
            }
            mbar_arrive_expect_tx(&ctl->full[slot], C::kSlotBytes);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) return false;
        const int lp = lane / C::kChunks, lc = lane % C::kChunks;
        const int prc = __shfl_sync(0xffffffffu, rc, lp & 31);
        if (lp < pages) {
          uint8_t* dst = kv_s + slot * C::kSlotBytes + lc * (kKeys * 128) + ((uint32_t)lp << (log_r + 7));
          tma_load_3d(dst, tm, lc * 64, k, prc, &ctl->full[slot]);
        }
        ++n_loads;
        return true;
      };
      for (uint32_t tt = 0; ok; ++tt) {
        const int slot = tt % kInfoRing;
        int got = 1;
        if (lane == 0)
          got = wait_or_abort(&ctl->info_full[slot], (tt / kInfoRing) & 1, abort, p.err, p.err_site, kSiteTree | 4);
        if (!__shfl_sync(0xffffffffu, got, 0)) break;
        const Segment cur = ctl->seg[slot];
        if (!cur.live) break;
        const int end = cur.past + cur.n;
        const int* bt_row = p.block_table + (size_t)cur.b * p.MB;
        auto load_id = [&](int e) -> int {
          return (e < p.MB && ((long long)e << p.log_bs) < end) ? bt_row[e] : -1;
        };
        int win = cur.key0 >> p.log_bs;
        int id = load_id(win + lane);
        for (int i = 0; i < cur.nt; ++i) {
          const int key0 = cur.key0 + i * kKeys;
          if (((key0 + kKeys - 1) >> p.log_bs) >= win + 32) {
            win = key0 >> p.log_bs;
            id = load_id(win + lane);
          }
          const int pos = key0 + (lane << log_r);
          const int idx = (pos >> p.log_bs) - win;
          const int blk = __shfl_sync(0xffffffffu, id, idx & 31);
          int rc = p.oob_row;
          if (lane < pages && pos < end) {
            if (blk >= 0 && blk < p.NB) rc = (blk << p.log_bs) + (pos & (p.bs - 1));
            else if (blk != -1) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
          }
          const uint32_t mask = __ballot_sync(0xffffffffu, lane < pages && rc == p.oob_row);
          if (!load_tile(&tm_k, cur.k, rc, false, mask) || !load_tile(&tm_v, cur.k, rc, true, 0)) break;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&ctl->info_empty[slot]);
      }
      if (lane == 0 && *abort) {
        for (int d = 1; d <= S && (int)n_loads - d >= 0; ++d) {
          const uint32_t n = n_loads - d;
          for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&ctl->full[n % S], (n / S) & 1); ++i) {
          }
        }
      }
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------- MMA issuer
      // A segment's jobs j = 0, 1, ... alternate between the streams: job j
      // is stream j & 1 and key tile j / 2 (two row tiles) or j (one).  In
      // issue order S(0) S(1) PV(0) S(2) PV(1) S(3) ...: S(j + 2) may
      // overwrite P(j)'s columns because MMAs of one thread complete in order,
      // and a wait on S(j + 2) covers PV(j).
      constexpr uint32_t idesc_s = umma_idesc_f16(kRows, kKeys, 0, 0, BF ? 1 : 0);
      constexpr uint32_t idesc_o = umma_idesc_f16(kRows, D, 0, 1, BF ? 1 : 0);
      const uint64_t desc_k = smem_desc_sw128(0, 16, 1024);           // K-major Q and K, + (address >> 4)
      const uint64_t desc_v = smem_desc_sw128(0, kKeys * 128, 1024);  // MN-major V, + (address >> 4)
      const uint32_t kv_addr = smem_u32(kv_s), q_addr = smem_u32(q_s);
      const bool leader = elect_one();
      auto wait_bar = [&](uint64_t* bar, uint32_t parity) -> bool {
        return wait_or_abort(bar, parity, abort, p.err, p.err_site, kSiteTree | 5);
      };
      uint32_t g = 0, pcnt[2] = {0, 0};
      bool ok = leader;
      for (uint32_t tt = 0; ok; ++tt) {
        const int slot = tt % kInfoRing;
        if (!wait_bar(&ctl->info_full[slot], (tt / kInfoRing) & 1)) break;
        const Segment& sg = ctl->seg[slot];
        if (!sg.live) break;
        const int two = sg.two, nt = sg.nt, jobs = two ? 2 * nt : nt;
        auto issue_s = [&](int j) -> bool {
          const int X = j & 1, i = two ? j >> 1 : j;
          const uint32_t n = 2 * (g + i);
          const int st = n % S;
          if (j == 0 && !wait_bar(&ctl->q_full, tt & 1)) return false;
          if ((!two || X == 0) && !wait_bar(&ctl->full[st], (n / S) & 1)) return false;
          tc_fence_after();
          const uint64_t a0 = desc_k + ((q_addr + (two ? X : 0) * C::kQTileBytes) >> 4);
          const uint64_t b0 = desc_k + ((kv_addr + st * C::kSlotBytes) >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_f16(tmem + C::s_col(X), a0 + (((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4),
                     b0 + (((ks >> 2) * (kKeys * 128) + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
          umma_commit(&ctl->s_full[X]);
          if (!two || X == 1) umma_commit(&ctl->empty[st]);
          if (j == jobs - 1) umma_commit(&ctl->q_empty);
          return true;
        };
        auto issue_pv = [&](int j) -> bool {
          const int X = j & 1, i = two ? j >> 1 : j;
          if (!wait_bar(&ctl->p_full[X], pcnt[X] & 1)) return false;
          ++pcnt[X];
          // the segment's first PV of the stream overwrites O_X: the last segment's has been read
          if (j < 2 && tt > 0 && !wait_bar(&ctl->o_free[X], (tt - 1) & 1)) return false;
          const uint32_t n = 2 * (g + i) + 1;
          const int st = n % S;
          if ((!two || X == 0) && !wait_bar(&ctl->full[st], (n / S) & 1)) return false;
          tc_fence_after();
          const uint64_t b0 = desc_v + ((kv_addr + st * C::kSlotBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_f16_ts(tmem + C::o_col(X), tmem + C::s_col(X) + kk * 8, b0 + ((kk * 16 * 128) >> 4), idesc_o,
                        (j > 1 || kk > 0) ? 1u : 0u);
          if (!two || X == 1) umma_commit(&ctl->empty[st]);
          if (j >= jobs - 2) umma_commit(&ctl->o_done[X]);
          return true;
        };
        ok = issue_s(0) && (jobs == 1 || issue_s(1));
        for (int j = 0; j < jobs && ok; ++j) ok = issue_pv(j) && (j + 2 >= jobs || issue_s(j + 2));
        g += nt;
        if (!ok) break;
        mbar_arrive(&ctl->info_empty[slot]);
      }
      // Drain: every MMA issued above has completed before TMEM is freed.
      if (leader) {
        umma_commit(&ctl->drain);
        for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&ctl->drain, 0); ++i) {
        }
      }
      __syncwarp();
    }
  } else {
    regs_inc<kRegSoftmax>();
    // ------------------------------------------- softmax and epilogue warps
    const int X = warp >> 2;            // stream
    const int r = threadIdx.x & 127;    // row of the tile == TMEM lane
    const int rj = r / p.G;             // its token within the tile
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float mul = GEN ? 1.f : p.scale * kLog2e;
    uint32_t g = 0, scnt = 0, ocnt[2] = {0, 0};
    float x[kKeys];
    for (uint32_t tt = 0;; ++tt) {
      const int slot = tt % kInfoRing;
      if (!wait_or_abort(&ctl->info_full[slot], (tt / kInfoRing) & 1, abort, p.err, p.err_site, kSiteTree | 6)) break;
      const Segment& sg = ctl->seg[slot];
      if (!sg.live) break;
      // the exchange of the last segment has been read by both streams
      if (tt > 0 && !wait_or_abort(&ctl->xchg_done, (tt - 1) & 1, abort, p.err, p.err_site, kSiteTree | 7)) break;
      const int two = sg.two, nt = sg.nt, past = sg.past, n = sg.n;
      const int jt = (two ? X * p.tile_tokens : 0) + rj;  // the row's token within the unit
      const bool row_ok = rj < p.tile_tokens && jt < sg.ntok;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int t = sg.t0 + (row_ok ? jt : 0);
      const int j_seq = t - sg.seq_t0;  // its draft index
      int qpos = 0, lo_row = 0;
      float slope2 = 0.f;
      if constexpr (GEN) {
        qpos = p.positions ? p.positions[t] : past + j_seq;
        if (p.window >= 1) lo_row = max(max(qpos, past) - p.window + 1, 0);
        if (p.slopes && row_ok) slope2 = p.slopes[sg.k * p.G + (r - rj * p.G)] * kLog2e;
      }
      const int lo_min = GEN && p.window >= 1 ? max(0, past + 1 - p.window) : 0;  // no row admits a key below
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = two ? 0 : X; i < nt; i += two ? 1 : 2) {
        const uint32_t nv = 2 * (g + i) + 1, tile = g + i;
        const int sv = nv % S;
        const int key0 = sg.key0 + i * kKeys;
        // (published before the tile's K load: read before the wait for S,
        // which hides the shared-memory load)
        if (!wait_or_abort(&ctl->mask_full[tile % kMaskRing], (tile / kMaskRing) & 1, abort, p.err, p.err_site,
                           kSiteTree | 8)) {
          ok = false;
          break;
        }
        const uint32_t pmask = ctl->kv_mask[tile % kMaskRing];
        if (!wait_or_abort(&ctl->s_full[X], scnt & 1, abort, p.err, p.err_site, kSiteTree | 9)) {
          ok = false;
          break;
        }
        const bool first = i == (two ? 0 : X);
        ++scnt;
        tc_fence_after();
        if (warp_ok) {
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) tmem_ld32(lane_addr + C::s_col(X) + c, x + c);
          tmem_ld_wait();
          if constexpr (GEN) {
            if (p.softcap > 0.f) {
              // c tanh(y) = c (1 - 2 / (1 + e^{2y})), in log2 units
              const float in = 2.f * kLog2e * p.scale / p.softcap, out = p.softcap * kLog2e;
#pragma unroll
              for (int c = 0; c < kKeys; ++c) x[c] = fmaf(-2.f * out, __frcp_rn(1.f + ex2(x[c] * in)), out);
            } else {
              const float in = p.scale * kLog2e;
#pragma unroll
              for (int c = 0; c < kKeys; ++c) x[c] *= in;
            }
            if (p.slopes) {
              const float base = (float)((long long)key0 - qpos);
              if (key0 + kKeys <= past || !p.positions) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c) x[c] = fmaf(slope2, base + (float)c, x[c]);
              } else {
#pragma unroll
                for (int c = 0; c < kKeys; ++c) {
                  const int d = key0 + c - past;  // draft index
                  const float gap = d < 0 || d >= n ? base + (float)c
                                                    : (float)((long long)p.positions[sg.seq_t0 + d] - qpos);
                  x[c] = fmaf(slope2, gap, x[c]);
                }
              }
            }
          }
          if (key0 + kKeys > past || key0 < lo_row || pmask != 0 || !row_ok) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k0 = key0 + 32 * q;
              uint32_t w = 0;
              if (row_ok) {
                w = bit_range(lo_row - k0, past - k0);
                const int d0 = k0 - past;  // draft index of bit 0
                if (d0 + 32 > 0 && d0 < n) {
                  uint32_t w2;
                  if (p.mask) {
                    const uint32_t* row = p.mask + (size_t)t * p.words;
                    const int wi = d0 >> 5;  // (floor)
                    const uint32_t a = wi >= 0 && wi < p.words ? row[wi] : 0u;
                    const uint32_t b = wi + 1 >= 0 && wi + 1 < p.words ? row[wi + 1] : 0u;
                    w2 = __funnelshift_r(a, b, d0 & 31);
                  } else {
                    w2 = bit_range(0, j_seq + 1 - d0);
                  }
                  w2 &= bit_range(-d0, n - d0);
                  if constexpr (GEN) {
                    if (p.window >= 1) {
                      for (int e = max(0, -d0); e < min(32, n - d0); ++e) {
                        const int kpos = p.positions ? p.positions[sg.seq_t0 + d0 + e] : past + d0 + e;
                        if (kpos < lo_row) w2 &= ~(1u << e);
                      }
                    }
                  }
                  w |= w2;
                }
                if (pmask != 0) {
                  for (int g2 = 0; g2 < pages; ++g2)
                    if ((pmask >> g2) & 1) w &= ~bit_range((g2 << log_r) - 32 * q, ((g2 + 1) << log_r) - 32 * q);
                }
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) x[32 * q + e] = ((w >> e) & 1) ? x[32 * q + e] : -INFINITY;
            }
          }
          const float cand = max_tree<kKeys>(x) * mul;
          float alpha = 1.f;
          if (cand > m_ref + kLazyRescale || (m_ref == -INFINITY && cand != -INFINITY)) {
            alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - cand);
            m_ref = cand;
          }
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t mul2 = f2(mul, mul), neg_m2 = f2(-m_use, -m_use);
          uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int h = 0; h < kKeys; h += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const uint64_t arg = fma2(f2(x[h + 2 * q], x[h + 2 * q + 1]), mul2, neg_m2);
              float a0, a1;
              unf2(arg, a0, a1);
              const float e0 = ex2(a0), e1 = ex2(a1);
              sum2[q & 3] = add2(sum2[q & 3], f2(e0, e1));
              pk[q] = pack2<BF>(e0, e1);
            }
            // P -> TMEM over S: keys h..h+31 as 16 columns of 16-bit pairs
            tmem_st16(lane_addr + C::s_col(X) + h / 2, pk);
          }
          if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
            float o[32];
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld32(lane_addr + C::o_col(X) + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(lane_addr + C::o_col(X) + 32 * c, o);
            }
          }
          float s0, s1, s2, s3;
          unf2(add2(sum2[0], sum2[1]), s0, s1);
          unf2(add2(sum2[2], sum2[3]), s2, s3);
          l = l * alpha + ((s0 + s1) + (s2 + s3));
        }
        // Zero V rows that no row admits by position, take non-finite values
        // out of draft rows (once per tile: stream 0 when both use it).
        if ((key0 + kKeys > past || key0 < lo_min) && (!two || X == 0)) {
          uint8_t* vs = kv_s + sv * C::kSlotBytes;
          if (!wait_or_abort(&ctl->full[sv], (nv / S) & 1, abort, p.err, p.err_site, kSiteTree | 10)) {
            ok = false;
            break;
          }
          for (int idx = r; idx < kKeys * C::kChunks * 8; idx += 128) {
            const int kr = idx / (C::kChunks * 8), rem = idx % (C::kChunks * 8);
            const int pos = key0 + kr;
            uint4* at = reinterpret_cast<uint4*>(vs + (rem >> 3) * (kKeys * 128) + kr * 128 +
                                                 (((rem & 7) ^ (kr & 7)) << 4));
            if (pos >= past + n || pos < lo_min) {
              *at = make_uint4(0, 0, 0, 0);
            } else if (pos >= past) {
              const uint4 v = *at;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              bool any = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (nonfinite16<BF>(w[e])) { w[e] &= 0xffff0000u; any = true; }
                if (nonfinite16<BF>(w[e] >> 16)) { w[e] &= 0x0000ffffu; any = true; }
              }
              if (any) {
                *at = make_uint4(w[0], w[1], w[2], w[3]);
                atomicOr(&ctl->bad[warp][(pos - past) >> 5], 1u << ((pos - past) & 31));
              }
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[X]);
      }
      if (!ok) break;

      // ---- end of the segment: the streams show each other their maxima and
      // sums (needed when they hold the same rows), then O leaves TMEM.
      ctl->ml[X][r] = make_float2(m_ref, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->xchg_full);
      if (!wait_or_abort(&ctl->xchg_full, tt & 1, abort, p.err, p.err_site, kSiteTree | 11)) break;
      float f0 = 1.f, f1 = 1.f;  // factors of O_0 and O_1 (one row tile)
      if (!two) {
        const float2 a = ctl->ml[0][r], b = ctl->ml[1][r];
        m_ref = fmaxf(a.x, b.x);
        f0 = a.x == -INFINITY ? 0.f : ex2(a.x - m_ref);
        f1 = b.x == -INFINITY ? 0.f : ex2(b.x - m_ref);
        l = (f0 == 0.f ? 0.f : f0 * a.y) + (f1 == 0.f ? 0.f : f1 * b.y);
      }
      uint32_t bad[kTreeMaxWords], any_bad = 0;
#pragma unroll
      for (int q = 0; q < kTreeMaxWords; ++q) {
        bad[q] = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) bad[q] |= ctl->bad[w][q];
        any_bad |= bad[q];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->xchg_done);
      if (any_bad) {
        // cleared for the next segment once both streams have read it
        if (!wait_or_abort(&ctl->xchg_done, tt & 1, abort, p.err, p.err_site, kSiteTree | 12)) break;
        if (lane < kTreeMaxWords) ctl->bad[warp][lane] = 0;
        __syncwarp();
      }
      const int jobs = two ? 2 * nt : nt;
      bool have[2] = {true, jobs >= 2};
      for (int Y = 0; Y < 2 && ok; ++Y) {
        if (!have[Y]) continue;
        if ((!two || Y == X) &&
            !wait_or_abort(&ctl->o_done[Y], ocnt[Y] & 1, abort, p.err, p.err_site, kSiteTree | 13))
          ok = false;
        ++ocnt[Y];
      }
      if (!ok) break;
      tc_fence_after();
      const int h = sg.k * p.G + (r - rj * p.G);
      float inv = 1.f;
      if (sg.slot < 0) {
        if (p.head_sink && row_ok && m_ref != -INFINITY)
          l += ex2(elem16_to_float(p.head_sink[h], BF) * kLog2e - m_ref);
        inv = l == 0.f ? 0.f : 1.f / l;
      }
      const int row = (two ? X * kRows : 0) + r;  // row of the unit's partial result
      if (sg.slot >= 0 && row_ok && (two || X == 0)) p.part_ml[(size_t)sg.slot * p.part_rows + row] = make_float2(m_ref, l);
      __half* dst = p.out + ((size_t)t * p.H + h) * D;
      float4* part = sg.slot >= 0 ? p.part_o + (size_t)sg.slot * (D / 4) * p.part_rows + row : nullptr;
      // two row tiles: every channel of the own O; one: half the channels of both
      const int c0 = two ? 0 : X * (D / 64), c1 = two ? D / 32 : (X + 1) * (D / 64);
      if (warp_ok) {
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float o[32];
          tmem_ld32(lane_addr + C::o_col(two ? X : 0) + 32 * c, o);
          if (!two) {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = f0 == 0.f ? 0.f : o[e] * f0;
            if (have[1]) {
              tmem_ld32(lane_addr + C::o_col(1) + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = f1 == 0.f ? o[e] : fmaf(x[e], f1, o[e]);
            }
          } else {
            tmem_ld_wait();
          }
          if (any_bad && row_ok) {
            for (int i = 0; i < n; ++i) {
              if (!((bad[i >> 5] >> (i & 31)) & 1) || !mask_bit(p, t, j_seq, i)) continue;
              if constexpr (GEN) {
                const int kpos = p.positions ? p.positions[sg.seq_t0 + i] : past + i;
                if (p.window >= 1 && kpos < lo_row) continue;
              }
              const int pos = past + i;
              const int blk = p.block_table[(size_t)sg.b * p.MB + (pos >> p.log_bs)];
              if (blk < 0 || blk >= p.NB) continue;
              const __half* v = p.value_cache +
                                ((((size_t)blk << p.log_bs) + (pos & (p.bs - 1))) * p.Hk + sg.k) * D + 32 * c;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (nonfinite16<BF>(__half_as_ushort(v[e]))) o[e] += elem16_to_float(v[e], BF);
            }
          }
          if (row_ok) {
            if (part) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                part[(size_t)(8 * c + q) * p.part_rows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint4 w;
                w.x = pack2<BF>(o[8 * q + 0] * inv, o[8 * q + 1] * inv);
                w.y = pack2<BF>(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
                w.z = pack2<BF>(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
                w.w = pack2<BF>(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
                *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = w;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->o_free[0]);
        mbar_arrive(&ctl->o_free[1]);
        mbar_arrive(&ctl->info_empty[slot]);
      }
      g += nt;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the partial results of the units that range borders cut: block
// (c, y) takes rows 32y.. of the unit that starts in CTA c's range.  A lane
// is a row, a warp 8 channels: partials are stored channel group by channel
// group with rows side by side, so both kernels access them coalesced.
template <int D, bool BF>
__global__ void __launch_bounds__(D / 8 * 32) tree_join_kernel(const __grid_constant__ TreeParams p) {
  griddep_wait();
  const Cut cut = p.cuts[blockIdx.x];
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), c8 = threadIdx.x >> 5;
  if (row >= cut.rows) return;
  const int X = row / kRows, r = row - X * kRows, rj = r / p.G, j = X * p.tile_tokens + rj;
  if (rj >= p.tile_tokens || j >= cut.ntok) return;
  const int t = cut.t0 + j, h = cut.k * p.G + (r - rj * p.G);
  const int ns = cut.more + 1;
  auto slot_of = [&](int s) -> size_t { return s == 0 ? cut.slot0 : 2 * (blockIdx.x + s); };
  float M = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < ns; ++s) M = fmaxf(M, p.part_ml[slot_of(s) * p.part_rows + row].x);
  float den = 0.f, acc[8] = {};
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const size_t at = slot_of(s);
    const float2 ml = p.part_ml[at * p.part_rows + row];
    const float4* o = p.part_o + (at * (D / 4) + 2 * c8) * p.part_rows + row;
    const float4 a = o[0], b = o[p.part_rows];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    if (f != 0.f) {
      den += f * ml.y;
      acc[0] += f * a.x; acc[1] += f * a.y; acc[2] += f * a.z; acc[3] += f * a.w;
      acc[4] += f * b.x; acc[5] += f * b.y; acc[6] += f * b.z; acc[7] += f * b.w;
    }
  }
  if (p.head_sink && M != -INFINITY) den += ex2(elem16_to_float(p.head_sink[h], BF) * kLog2e - M);
  const float inv = den == 0.f ? 0.f : 1.f / den;
  *reinterpret_cast<uint4*>(p.out + ((size_t)t * p.H + h) * D + 8 * c8) =
      make_uint4(pack2<BF>(acc[0] * inv, acc[1] * inv), pack2<BF>(acc[2] * inv, acc[3] * inv),
                 pack2<BF>(acc[4] * inv, acc[5] * inv), pack2<BF>(acc[6] * inv, acc[7] * inv));
}

template <int D, bool BF, bool GEN>
cudaError_t configure() {
  using C = TreeCfg<D>;
  static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");
  static_assert(C::kSmemBytes <= kSmemLimit, "shared memory");
  static_assert(C::kSlots >= 4, "K/V ring");
  static_assert(2 * kKeys + 2 * D <= C::kTmemCols, "tensor memory");
  return cudaFuncSetAttribute(tree_kernel<D, BF, GEN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
}

template <int D, bool BF>
cudaError_t configure_db() {
  const cudaError_t e = configure<D, BF, false>();
  return e != cudaSuccess ? e : configure<D, BF, true>();
}

template <int D, bool BF>
cudaError_t launch_db(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                      int grid, cudaStream_t s) {
  const bool gen = p.softcap > 0.f || p.slopes || p.window >= 1;
  cudaError_t e = gen ? launch_pdl(tree_kernel<D, BF, true>, dim3(grid), kThreads, TreeCfg<D>::kSmemBytes, s, tq, tk,
                                   tv, p)
                      : launch_pdl(tree_kernel<D, BF, false>, dim3(grid), kThreads, TreeCfg<D>::kSmemBytes, s, tq, tk,
                                   tv, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_join_kernel<D, BF>, dim3(grid, (p.part_rows + 31) / 32), D / 8 * 32, 0, s, p);
}

}  // namespace

cudaError_t tree_configure(int head_size, int bf16) {
  if (head_size == 64) return bf16 ? configure_db<64, true>() : configure_db<64, false>();
  return bf16 ? configure_db<128, true>() : configure_db<128, false>();
}

cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                        int bf16, int grid, cudaStream_t s) {
  if (p.D == 64) return bf16 ? launch_db<64, true>(tq, tk, tv, p, grid, s) : launch_db<64, false>(tq, tk, tv, p, grid, s);
  return bf16 ? launch_db<128, true>(tq, tk, tv, p, grid, s) : launch_db<128, false>(tq, tk, tv, p, grid, s);
}

}  // namespace pa
