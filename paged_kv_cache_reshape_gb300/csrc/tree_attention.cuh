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
// length is its number of 128-key tiles plus a few that stand for its fixed
// cost.  The units of one kv head stand in a line (the same line for every
// head) that is cut into equal ranges, whatever unit borders they cross; a
// chunk is a range of one head, and consecutive chunks are the heads of one
// range, so that CTAs working at the same time read the same pool rows (one
// row holds all heads).  A CTA (one per SM) takes one chunk, or every
// gridDim-th.  A unit that a border cuts leaves partial results, which a
// second small kernel joins.  Every CTA lays out the line from the lengths by
// itself (one read of the lengths and a block scan), so the step needs no
// planning launch.
//
// A unit of two row tiles runs them as two streams over the same key tiles;
// a unit of one row tile runs its even and odd key tiles as the two streams
// and joins them at its end, so that either way one stream's softmax overlaps
// the other's tensor work.  Per stream: S and O in tensor memory (S = M 128 x
// N 128 columns, O = head_size columns), P over S as 16-bit pairs, read from
// there by the P V product.
//
// head_size 256: two O would not fit in tensor memory and 128-key tiles not in
// the ring, so a unit has one row tile, key tiles are 64 keys, and one stream
// (warpgroup 0) works through them with S double-buffered; the K/V bytes of a
// tile still cover its softmax.
//
// Few rows (head_size 64, at most 64 or 32): the row tile holds every row 2 or
// 4 times (REP), each replica takes the softmax of its own half or quarter of
// a tile's keys (its P is zero at the others), and the replicas' O, m and l
// are joined in shared memory at the segment's end: otherwise one or two
// warps of four would do all the exponentials.
//
// Masks: an interior tile (context only) needs none.  A tile that holds
// draft tokens, a window's edge or an unmapped page builds one 128-bit mask
// per row.  P is zero at masked keys, and 0 * inf would still be NaN in the
// P V product, so V rows past the sequence are zeroed in shared memory, and
// non-finite values in keys that only some rows admit (drafts, the context at
// a window's edge) are taken out there and added to the rows that do admit
// them when O leaves tensor memory.
//
// Roles (384 threads): warpgroups 0 and 1, softmax and epilogue of the two
// streams (thread = row = TMEM lane); warps 8 and 11 K and V producers (TMA,
// one ring of slots in the order of their use), warp 9 TMEM owner and MMA
// issuer, warp 10 takes chunks, publishes their segments and loads Q.
//
// What bounds it (one GB300; 6780 GB/s copied, 1925 TFLOP/s in a plain 16-bit
// matrix product; calls with their join, inputs not in L2):
//   64 sequences, 512..4096 keys, 8 tokens, 32/8 heads of 128   95 us  5.7 TB/s  the K/V stream
//   2 sequences, 100000..131072 keys, 32 tokens, 32/8 heads    145 us  6.2 TB/s  the K/V stream
//   16 sequences, 1024..8192 keys, 64 tokens, 64/8 heads       138 us  1.12 PFLOP/s in a few dozen calls;
//                            146 to 151 us, 1.02 to 1.06 PFLOP/s, in a thousand: the power cap lowers the clock
// The last is bound by each stream's chain S -> softmax -> P -> PV (2.0 us for
// a key tile of both streams, 1.1 us of it tensor work): the tensor pipe is
// active 57 % of the time, no other pipe above 30 %.  What did not help: P
// handed over in two halves (1.74 us a tile in a traced copy, but the call 144
// us against 141); at head_size 64 columns of its own for P, so that S runs two
// tiles ahead (121 against 117 us); the MMA issuer as a whole warp with an
// elected lane per batch (152 us); the softmax over 32 columns at a time, read
// twice from tensor memory (half the code; 146 us, with a cap 251 against 227).
// What the layout above is worth at the 64 sequences: consecutive chunks by
// head rather than by range 158 -> 109 us together with one 5-D box per page;
// K and V from two warps 109 -> 99 us; row replicas (head_size 64, bias) 75 ->
// 52 us; the equal static ranges against a queue of small chunks, at the 2
// long sequences, 142 against 154 us.  One sequence of 600 keys and 5 tokens
// takes 12 us, latency throughout: 3 us to the first S, 3 us for the join.
//
// Code size counts: one CTA per SM runs six different roles, and a segment's
// end is run once per segment by each.  Rarely run loops are therefore not
// unrolled and waits kept small: with 128 KB of code a segment's end took 4 to
// 7 us of instruction fetches, with 65 KB 1.5 us.
#include <algorithm>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "step.h"
#include "tree.h"

namespace pa {
namespace {

constexpr int kThreads = 12 * 32;
constexpr int kKWarp = 8, kMmaWarp = 9, kFetchWarp = 10, kVWarp = 11;
constexpr int kControlWarp0 = 8;
// Registers per thread after the split (launch: 168 each).
constexpr int kRegSoftmax = 208, kRegControl = 80;
static_assert(2 * kRegSoftmax + kRegControl <= 3 * 168, "register split");
constexpr int kRows = 128;   // rows per row tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyRescale = 8.f;  // log2 of the largest P value tolerated before rescaling
constexpr int kSmemLimit = 227 * 1024;
constexpr int kCtrlBytes = 3 * 1024;
constexpr int kInfoRing = 4;  // segments published ahead of their use
// Page masks of the K/V tiles in flight: the producer cannot be a whole ring
// ahead of a stream (a slot is reused only after MMAs that follow the softmax
// of all older tiles but the last few).
constexpr int kMaskRing = 16;
constexpr int kMaxSlots = 12;  // K/V ring slots at most
constexpr int kJoinChannels = 16;  // channels of the replicas joined at a time
// A unit's fixed cost in key tiles (64 sequences of 512..4096 keys with 0, 1,
// 2, 3: 100.1, 99.1, 97.3, 97.0 us when first swept; 95.6 with 2, 96.6 with 3 since).
constexpr int kUnitCost = 2;
constexpr int kMaxLen = 1 << 26;  // of a sequence in the line (a window of 32 stays below 2^31)
constexpr int kMinRange = 2;  // a line of less than twice this stays whole (2 was the best of a sweep)

template <int D>
struct TreeCfg {
  static constexpr bool kOneO = D == 256;          // one stream
  static constexpr int kKeys = kOneO ? 64 : 128;   // keys per K/V tile
  static constexpr int kChunks = D / 64;
  static constexpr int kQTileBytes = kRows * D * 2;  // [chunk][row][128 B]
  static constexpr int kSlotBytes = kKeys * D * 2;   // one K or V tile [key / 8][chunk][key % 8][128 B]
  static constexpr int kGroupBytes = kChunks * 1024;  // its 8-key groups
  // Slots of the K/V ring beside `q_tiles` Q tiles.
  static __host__ __device__ constexpr int slots(int q_tiles, int rep) {
    const int fit = (kSmemLimit - kCtrlBytes - join_bytes(rep) - q_tiles * kQTileBytes) / kSlotBytes;
    return fit < kMaxSlots ? fit : kMaxSlots;
  }
  // Where replicas are joined: per stream 128 lanes x 16 channels, and (m, l) per row.
  static __host__ __device__ constexpr int join_bytes(int rep) {
    return rep > 1 ? 2 * kRows * kJoinChannels * 4 + 2 * kRows * 8 : 0;
  }
  static __host__ __device__ constexpr int s_col(int X) { return X * kKeys; }
  static __host__ __device__ constexpr int o_col(int X) { return 2 * kKeys + (kOneO ? 0 : X * D); }
  static constexpr int kTmemCols = 512;
  // Whether V's slot may be waited for before S is also where tiles alternate (see mend_v).
  static __host__ __device__ constexpr bool v_ordered(int rep) { return kOneO ? slots(1, rep) >= 5 : slots(2, rep) >= 7; }
  static __host__ __device__ constexpr int smem_bytes(int q_tiles, int rep) {
    return q_tiles * kQTileBytes + slots(q_tiles, rep) * kSlotBytes + kCtrlBytes + join_bytes(rep);
  }
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
  float2 ml[2][kRows];                // per stream: running maximum and sum of the segment
  // Per segment parity: keys with non-finite V, first the draft tokens, then
  // the context from the window's edge `lo_min` on.
  uint32_t bad[2][2 * kTreeMaxWords];
  // Per stream, where replicas are joined: whether an output became NaN beside
  // a sum that is a number, and the channels with a +inf, -inf, NaN value.
  uint32_t lost[2], found[2][3];
  uint8_t kv_mask[kMaskRing];         // per K/V tile (tile number mod ring): its pages that are unmapped
  uint64_t mask_full[kMaskRing];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t pv_done;                   // one stream: after every PV
  uint64_t info_full[kInfoRing], info_empty[kInfoRing];
  uint64_t xchg_full, xchg_done, join[2];
  uint64_t drain;
  int scan[kThreads / 32];            // lengths of the first groups of 32 sequences, then where they start
  int total;                          // length of the line
  uint32_t tmem_base;
  int abort;
};

// A position in the K/V ring: the slot and the phase of its barriers.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// What the schedule needs of a sequence.
struct SeqWork {
  int past, n, t0;
  int lo;        // first key walked (a multiple of 128)
  int nt;        // key tiles of each unit
  int pairs;     // units
  int len;       // their length in the line
};

template <int kKeys>
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
    s.pairs = (((s.n - 1) * p.inv_unit) >> 20) + 1;  // ceil(n / unit_tokens)
    const long long len = (long long)(s.nt + kUnitCost) * s.pairs;
    if (len < kMaxLen) s.len = (int)len;
    else bits |= PA_DEVERR_KV_BOUND;
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

// Bounded mbarrier wait: gives up (returns false) when another role has set
// *abort, or after kWaitLimit polls, setting it to the wait's site.  (Small,
// for the code size.)
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int site) {
  uint32_t i = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (++i == kWaitLimit) *abort = kSiteTree | site;
    if ((i & 1023) == 0 && *abort) return false;
  }
  return true;
}

template <bool BF>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
  return BF ? (h & 0x7f80u) == 0x7f80u : (h & 0x7c00u) == 0x7c00u;
}
// The same for both halves of w, at bits 15 and 31: an exponent of all ones
// carries into the sign's place.
template <bool BF>
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w) {
  return (BF ? (w & 0x7f807f80u) + 0x00800080u : (w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// GEN: softcap, distance bias or a window (checked at run time); without it
// the scores need one multiplication.  REP: replicas of the rows.
template <int D, bool BF, bool GEN, int REP>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  constexpr int kKeys = C::kKeys;
  static_assert(REP == 1 || D == 64, "replicated rows");
  const int S = C::slots(p.q_tiles, REP);
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_s = smem;                                // [tile A (, tile B)]
  uint8_t* kv_s = q_s + p.q_tiles * C::kQTileBytes;  // [slot]
  Ctrl* ctl = reinterpret_cast<Ctrl*>(kv_s + S * C::kSlotBytes);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {  // the barriers, side by side
    if (lane < 2) {
      mbar_init(&ctl->s_full[lane], 1);
      mbar_init(&ctl->p_full[lane], 4);
      mbar_init(&ctl->o_done[lane], 1);
      mbar_init(&ctl->o_free[lane], 8);
      mbar_init(&ctl->join[lane], 4);
    } else if (lane < 2 + kInfoRing) {
      mbar_init(&ctl->info_full[lane - 2], 1);
      mbar_init(&ctl->info_empty[lane - 2], 1 + 8 + 2);  // MMA, softmax and K/V producer warps
    } else if (lane == 2 + kInfoRing) {
      mbar_init(&ctl->q_full, 1);
      mbar_init(&ctl->q_empty, 1);
      mbar_init(&ctl->xchg_full, 8);
      mbar_init(&ctl->xchg_done, 8);
      mbar_init(&ctl->drain, 1);
      mbar_init(&ctl->pv_done, 1);
      ctl->abort = 0;
    }
    if (lane < kMaskRing) {
      mbar_init(&ctl->mask_full[lane], 1);
    } else if (lane < kMaskRing + kMaxSlots) {
      mbar_init(&ctl->full[lane - kMaskRing], 1);
      mbar_init(&ctl->empty[lane - kMaskRing], 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x < 4 * kTreeMaxWords) ctl->bad[0][threadIdx.x] = 0;
  if (REP > 1 && threadIdx.x < 2) {
    ctl->lost[threadIdx.x] = 0;
    for (int i = 0; i < 3; ++i) ctl->found[threadIdx.x][i] = 0;
  }
  if (warp == kFetchWarp && lane == 0) prefetch_tmap(&tm_q);
  if (warp == kKWarp && lane == 0) prefetch_tmap(&tm_k);
  if (warp == kVWarp && lane == 0) prefetch_tmap(&tm_v);

  if ((smem_u32(smem) & 1023) != 0) {  // the swizzled operands need it; never seen
    if (threadIdx.x == 0) note_timeout(p.err, p.err_site, kSiteTree);
    return;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The allocation is all of tensor memory, so it starts at column 0: as a
  // constant the columns cost the MMA issuer and the softmax no registers
  // (16 sequences of 64 drafts 141 -> 138 us, short contexts 75 -> 69).
  constexpr uint32_t tmem = 0;
  static_assert(C::kTmemCols == 512, "tensor memory");

  griddep_wait();  // lengths, queries and pools may come from the previous kernel
  griddep_launch_dependents();

  // Where each group of 32 sequences starts in the line, and its length (a
  // batch of one group is left to the fetcher).
  int* const groups = p.batch <= kThreads ? ctl->scan : p.groups + (size_t)blockIdx.x * p.n_groups;
  if (p.n_groups > 1) {
    int bits = 0;
    long long before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      long long len = b < p.batch ? seq_work<kKeys>(p, b, bits).len : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) len += __shfl_xor_sync(0xffffffffu, len, o);
      // (no sum over a line of at most 2^31 - 1 wraps; a longer one is refused below)
      __syncthreads();
      if (lane == 0) ctl->scan[warp] = (int)min(len, 0x7fffffffll);
      __syncthreads();
      long long first = before;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) first += ctl->scan[w];
        before += ctl->scan[w];
      }
      if (p.batch <= kThreads) __syncthreads();  // the groups' starts replace their lengths
      if (lane == 0 && (b0 >> 5) + warp < p.n_groups) groups[(b0 >> 5) + warp] = (int)first;
    }
    if (before > 0x7fffffffll) {  // 2^31 key tiles: over ten seconds of work
      bits |= PA_DEVERR_KV_BOUND;
      before = 0;
    }
    if (bits && blockIdx.x == 0) atomicOr(p.err, bits);
    if (threadIdx.x == 0) ctl->total = (int)before;
    __syncthreads();
  }
  const int log_r = p.log_page_rows;  // log2(min(block_size, 128))
  const int pages = kKeys >> log_r;

  // Register split: each warpgroup resizes at the top of its own branch
  // (the allocator budgets a branch from the setmaxnreg that dominates it).
  if (warp >= kControlWarp0) {
    regs_dec<kRegControl>();
    if (warp == kFetchWarp) {
      // ---------------------------------------------------------- fetcher
      // Takes chunks, publishes their segments and loads a segment's Q tiles
      // once the previous segment's S products are done.
      const uint32_t q_bytes = C::kChunks * p.G * p.tile_tokens * 128;  // of one box
      // A window of 32 sequences, one per lane: where each ends in the line.
      int group = -1, win_lo = 0, win_hi = 0, seq_end = 0;
      SeqWork mine{};
      auto load_window = [&](int& bits) {
        const int b = 32 * group + lane;
        mine = SeqWork{};
        if (b < p.batch) mine = seq_work<kKeys>(p, b, bits);
        seq_end = mine.len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, seq_end, o);
          if (lane >= o) seq_end += up;
        }
        seq_end += win_lo;
        win_hi = __shfl_sync(0xffffffffu, seq_end, 31);
      };
      int ignored = 0, total;
      if (p.n_groups > 1) {
        total = ctl->total;
      } else {
        int bits = 0;
        group = 0;
        load_window(bits);
        if (bits && blockIdx.x == 0) atomicOr(p.err, bits);
        total = win_hi;
      }
      const int n_ranges = min(p.n_ranges, total / kMinRange + 1);
      const int n_chunks = total > 0 ? n_ranges * p.Hk : 0;
      const int len_q = total / n_ranges, len_r = total - len_q * n_ranges;
      auto range_begin = [&](int i) -> int { return len_q * i + min(i, len_r); };  // the first len_r are one longer
      int chunk = (int)blockIdx.x - (int)gridDim.x, range = 0;
      int r = 0, r_begin = 0, r_end = 0;
      uint32_t q_loads = 0;
      for (uint32_t tt = 0;; ++tt) {
        Segment f{};
        Cut cut{};
        while (true) {
          if (r >= r_end) {  // next chunk
            chunk += gridDim.x;
            if (chunk >= n_chunks) break;
            range = chunk / p.Hk;
            r = r_begin = range_begin(range);
            r_end = range_begin(range + 1);
            continue;
          }
          if (r >= win_hi || r < win_lo || group < 0) {
            int g0 = r < win_lo ? 0 : max(group, 0), at = 0;
            for (;; g0 += 32) {
              const int g = g0 + lane;
              const unsigned le = __ballot_sync(0xffffffffu, g < p.n_groups && groups[min(g, p.n_groups - 1)] <= r);
              at = __popc(le);  // groups start in order
              if (at < 32) break;
            }
            group = at > 0 ? g0 + at - 1 : g0 - 1;
            win_lo = groups[group];
            load_window(ignored);
          }
          const int src = __ffs(__ballot_sync(0xffffffffu, r < seq_end)) - 1;
          SeqWork s;
          s.past = __shfl_sync(0xffffffffu, mine.past, src);
          s.n = __shfl_sync(0xffffffffu, mine.n, src);
          s.t0 = __shfl_sync(0xffffffffu, mine.t0, src);
          s.lo = __shfl_sync(0xffffffffu, mine.lo, src);
          s.nt = __shfl_sync(0xffffffffu, mine.nt, src);
          const int off = r - __shfl_sync(0xffffffffu, seq_end - mine.len, src);
          const int u = off / (s.nt + kUnitCost), tile0 = off - u * (s.nt + kUnitCost);
          if (tile0 >= s.nt) {  // the unit's fixed cost
            r += s.nt + kUnitCost - tile0;
            continue;
          }
          f.live = 1;
          f.b = 32 * group + src;
          if (lane == 0) prefetch_l1(p.block_table + (size_t)f.b * p.MB + ((s.lo + tile0 * kKeys) >> p.log_bs));
          f.k = chunk % p.Hk;
          f.t0 = s.t0 + u * p.unit_tokens;
          f.ntok = min(p.unit_tokens, s.n - u * p.unit_tokens);
          f.two = f.ntok > p.tile_tokens;
          f.seq_t0 = s.t0;
          f.n = s.n;
          f.past = s.past;
          f.key0 = s.lo + tile0 * kKeys;
          f.nt = min(s.nt - tile0, r_end - r);
          f.slot = f.nt == s.nt ? -1 : 2 * chunk + (r == r_begin ? 0 : 1);
          if (tile0 == 0 && f.nt < s.nt) {  // the unit goes on in later ranges
            cut.rows = f.two ? kRows + (f.ntok - p.tile_tokens) * p.G : f.ntok * p.G;
            cut.slot0 = f.slot;
            cut.slot1 = 2 * (chunk + p.Hk);
            cut.more = 0;
            while (range_begin(range + cut.more + 1) < r + s.nt) ++cut.more;
            cut.t0 = f.t0;
            cut.ntok = f.ntok;
            cut.k = f.k;
          }
          r += f.nt;
          break;
        }
        const int slot = tt % kInfoRing;
        bool ok = true;
        if (lane == 0) {
          if (!tree_wait(&ctl->info_empty[slot], ((tt / kInfoRing) & 1) ^ 1, abort, 1)) {
            ok = false;
          } else {
            ctl->seg[slot] = f;
            mbar_arrive(&ctl->info_full[slot]);
            if (f.live) {
              if (!tree_wait(&ctl->q_empty, (tt & 1) ^ 1, abort, 2)) {
                ok = false;
              } else {
                // both row tiles, or the one, or its replicas
                const int boxes = f.two ? 2 : REP;
                mbar_arrive_expect_tx(&ctl->q_full, boxes * q_bytes);
#pragma unroll 1
                for (int i = 0; i < boxes; ++i)
                  for (int c = 0; c < C::kChunks; ++c)
                    tma_load_3d(q_s + i * (f.two ? C::kQTileBytes : kRows / REP * 128) + c * (kRows * 128), &tm_q, c * 64,
                                f.k * p.G, f.t0 + (f.two ? i * p.tile_tokens : 0), &ctl->q_full);
                ++q_loads;
              }
            }
          }
        }
        if (f.live) {
          // what the softmax warps will read of the unit's rows, towards L1
          if (GEN && p.positions && 32 * lane < f.ntok) prefetch_l1(p.positions + f.t0 + 32 * lane);
          if (GEN && p.slopes && lane == 31) prefetch_l1(p.slopes + f.k * p.G);
          if (p.mask && f.key0 + f.nt * kKeys > f.past)
            for (int i = 32 * lane; i < f.ntok * p.words; i += 1024) prefetch_l1(p.mask + (size_t)f.t0 * p.words + i);
        }
        if (lane == 0 && cut.rows > 0) {  // units in two pieces from the front, in more from the back
          const int many = cut.more > 1, at = atomicAdd(&p.counters->n_cuts[many], 1);
          if (at < p.n_ranges * p.Hk) p.cuts[many ? p.n_ranges * p.Hk - 1 - at : at] = cut;
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok || !f.live) break;
      }
      if (lane == 0 && *abort && q_loads > 0) {
        // Gave up: let the copies already issued land before the CTA exits.
        for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&ctl->q_full, (q_loads - 1) & 1); ++i) {
        }
      }
    } else if (warp == kKWarp || warp == kVWarp) {
      // ---------------------------------------------------- K, V producers
      // Both walk the same loads (in the order of use, see the MMA issuer:
      // K_i V_i with two row tiles, K_i V_{i-1} with one) and issue their own.
      const bool v_warp = warp == kVWarp;
      const CUtensorMap* tm = v_warp ? &tm_v : &tm_k;
      uint32_t n_tiles = 0;             // tiles issued so far
      uint32_t issued = 0, phases = 0;  // per slot: loaded by this warp; the phase of that load
      RingPos at;
      bool ok = true;
      for (uint32_t tt = 0; ok; ++tt) {
        const int slot = tt % kInfoRing;
        int got = 1;
        if (lane == 0) got = tree_wait(&ctl->info_full[slot], (tt / kInfoRing) & 1, abort, 4);
        if (!__shfl_sync(0xffffffffu, got, 0)) break;
        const Segment cur = ctl->seg[slot];
        if (!cur.live) break;
        const int end = cur.past + cur.n;
        const int* bt_row = p.block_table + (size_t)cur.b * p.MB;
        auto load_id = [&](int e) -> int {
          return (e < p.MB && ((long long)e << p.log_bs) < end) ? bt_row[e] : -1;
        };
        // block ids of 32 pages, one per lane, and of the 32 behind them
        int win = cur.key0 >> p.log_bs;
        int id = load_id(win + lane), id_next = load_id(win + 32 + lane), rc = p.oob_row, rc_before = 0;
        const int lag = cur.two ? 0 : 1;
#pragma unroll 1
        for (int l = 0; l < 2 * (cur.nt + lag); ++l) {
          const bool is_v = l & 1;
          const int i = l >> 1;
          if (is_v ? i < lag : i >= cur.nt) continue;
          uint32_t mask = 0;
          if (!is_v) {  // the tile's pages
            const int key0 = cur.key0 + i * kKeys;
            if (((key0 + kKeys - 1) >> p.log_bs) >= win + 32) {
              win += 32;
              id = id_next;
              id_next = load_id(win + 32 + lane);
            }
            const int pos = key0 + (lane << log_r);
            const int idx = (pos >> p.log_bs) - win;
            const int blk = __shfl_sync(0xffffffffu, id, idx & 31);
            rc_before = rc;
            rc = p.oob_row;
            if (lane < pages && pos < end) {
              if (blk >= 0 && blk < p.NB) rc = (blk << p.log_bs) + (pos & (p.bs - 1));
              else if (blk != -1) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
            }
            mask = __ballot_sync(0xffffffffu, lane < pages && rc == p.oob_row);
          }
          if (is_v == v_warp) {  // into the ring's next slot, page by page
            const int row = is_v && lag && i < cur.nt ? rc_before : rc;
            uint8_t* const dst = kv_s + at.slot * C::kSlotBytes;
            const int step = C::kGroupBytes << (log_r - 3);  // of a page
            // One lane copies all pages, or lane l copies page l (the copies are
            // issued one after the other either way, from the lanes each with
            // operands of its own).  With 64 channels the issue of small pages
            // bounds the K/V stream and one lane is faster (pages of 16: 64
            // sequences 69.0 -> 63.3 us, two long ones 100 -> 91; of 32, wide
            // trees: 113.6 -> 116.7); with more channels the lanes are (64
            // sequences 95.5 against 96.7 us, two long ones 145.4 against 146.2).
            constexpr bool kOneLane = D == 64;
            int page_row[kKeys / 16];
            if constexpr (kOneLane) {
#pragma unroll
              for (int g = 0; g < kKeys / 16; ++g) page_row[g] = __shfl_sync(0xffffffffu, row, g);
            }
            if (kOneLane ? elect_one() : lane == 0) {
              if (!tree_wait(&ctl->empty[at.slot], at.phase ^ 1, abort, 3)) {
                ok = false;
              } else {
                if (!is_v) {
                  ctl->kv_mask[n_tiles % kMaskRing] = (uint8_t)mask;
                  mbar_arrive(&ctl->mask_full[n_tiles % kMaskRing]);
                }
                mbar_arrive_expect_tx(&ctl->full[at.slot], C::kSlotBytes);
                if constexpr (kOneLane) {
#pragma unroll
                  for (int g = 0; g < kKeys / 16; ++g)
                    if (g < pages) tma_load_5d(dst + g * step, tm, 0, 0, 0, page_row[g] >> 3, cur.k, &ctl->full[at.slot]);
                }
              }
            }
            ok = kOneLane ? __all_sync(0xffffffffu, ok) : __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (!kOneLane && lane < pages)
              tma_load_5d(dst + lane * step, tm, 0, 0, 0, row >> 3, cur.k, &ctl->full[at.slot]);
            issued |= 1u << at.slot;
            phases = (phases & ~(1u << at.slot)) | (at.phase << at.slot);
            ++n_tiles;
          }
          at.next(S);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&ctl->info_empty[slot]);
      }
      if (lane == 0 && *abort) {
        // Gave up: let the copies already issued land before the CTA exits.
        for (int i = 0; i < S; ++i)
          for (uint32_t k = 0; ((issued >> i) & 1) && k < kWaitLimit && !mbar_try_wait(&ctl->full[i], (phases >> i) & 1); ++k) {
          }
      }
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------- MMA issuer
      // A segment's jobs j = 0, 1, ... alternate between the streams: job j
      // is stream j & 1 and key tile j / 2 (two row tiles) or j (one).  In
      // issue order S(0) S(1) PV(0) S(2) PV(1) S(3) ...: S(j + 2) may
      // overwrite P(j)'s columns because MMAs of one thread complete in order,
      // and a wait on S(j + 2) covers PV(j).  First uses of tiles: with two
      // row tiles K0 V0 K1 V1 ..., with one K0 K1 V0 K2 V1 K3 ... (the ring's
      // order, so that a slot is free as soon as it is the next to be filled).
      constexpr int kFirstJobs = C::kOneO ? 1 : 2;  // jobs whose PV is the first into its O
      constexpr uint32_t idesc_s = umma_idesc_f16(kRows, kKeys, 0, 0, BF ? 1 : 0);
      constexpr uint32_t idesc_o = umma_idesc_f16(kRows, D, 0, 1, BF ? 1 : 0);
      const uint64_t desc_q = smem_desc_sw128(0, 16, 1024);                // K-major Q, + (address >> 4)
      const uint64_t desc_k = smem_desc_sw128(0, 16, C::kGroupBytes);      // K-major K
      const uint64_t desc_v = smem_desc_sw128(0, 1024, C::kGroupBytes);    // MN-major V
      const uint32_t kv_addr = smem_u32(kv_s), q_addr = smem_u32(q_s);
      const bool leader = elect_one();
      auto wait_bar = [&](uint64_t* bar, uint32_t parity) -> bool {
        return tree_wait(bar, parity, abort, 5);
      };
      uint32_t pcnt = 0;  // bit X: parity of p_full[X]
      RingPos at;
      int k_slot = 0, v_slot = 0;  // slots that the second row tile uses again
      bool ok = leader;
      for (uint32_t tt = 0; ok; ++tt) {
        const int slot = tt % kInfoRing;
        if (!wait_bar(&ctl->info_full[slot], (tt / kInfoRing) & 1)) break;
        const Segment& sg = ctl->seg[slot];
        if (!sg.live) break;
        const int two = sg.two, nt = sg.nt, jobs = two ? 2 * nt : nt;
#pragma unroll 1
        for (int j = 0; j < jobs + 2 && ok; ++j) {
          const int X = j & 1;
          if (j >= 2) {  // O_X += P_X V of job j - 2
            // its P; the segment's first PV of the stream overwrites O_X, which the last segment has read
            ok = wait_bar(&ctl->p_full[X], (pcnt >> X) & 1) &&
                 (j >= kFirstJobs + 2 || tt == 0 || wait_bar(&ctl->o_free[X], (tt - 1) & 1));
            if (!ok) break;
            pcnt ^= 1u << X;
            if (!two || X == 0) {
              if (!(ok = wait_bar(&ctl->full[at.slot], at.phase))) break;
              v_slot = at.slot;
              at.next(S);
            }
            tc_fence_after();
            const uint64_t b0 = desc_v + ((kv_addr + v_slot * C::kSlotBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_f16_ts(tmem + C::o_col(0) + (C::kOneO ? 0 : X * D), tmem + X * kKeys + kk * 8,
                          b0 + ((kk * 2 * C::kGroupBytes) >> 4), idesc_o, (j >= kFirstJobs + 2 || kk > 0) ? 1u : 0u);
            if (!two || X == 1) umma_commit(&ctl->empty[v_slot]);
            if constexpr (C::kOneO) {
              umma_commit(&ctl->pv_done);
              if (j == jobs + 1) umma_commit(&ctl->o_done[0]);
            } else {
              if (j >= jobs) umma_commit(&ctl->o_done[X]);
            }
          }
          if (j < jobs) {  // S_X = Q K^T of job j
            if (j == 0 && !(ok = wait_bar(&ctl->q_full, tt & 1))) break;
            if (!two || X == 0) {
              if (!(ok = wait_bar(&ctl->full[at.slot], at.phase))) break;
              k_slot = at.slot;
              at.next(S);
            }
            tc_fence_after();
            const uint64_t a0 = desc_q + ((q_addr + (two ? X : 0) * C::kQTileBytes) >> 4);
            const uint64_t b0 = desc_k + ((kv_addr + k_slot * C::kSlotBytes) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_f16(tmem + X * kKeys, a0 + (((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4),
                       b0 + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
            umma_commit(&ctl->s_full[X]);
            if (!two || X == 1) umma_commit(&ctl->empty[k_slot]);
            if (j == jobs - 1) umma_commit(&ctl->q_empty);
          }
        }
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
    constexpr int R = kRows / REP, COLS = kKeys / REP;
    const int r = threadIdx.x & 127;    // TMEM lane
    const int row = r & (R - 1);        // row of the tile
    const int cb = r / R * COLS;        // first of the tile's keys that this replica takes
    const int rj = row / p.G;           // the row's token within the tile
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float mul = (GEN && p.softcap > 0.f ? p.softcap : p.scale) * kLog2e;  // of x, to log2 units
    uint32_t g = 0, scnt = 0, ocnt[2] = {0, 0};
    uint32_t pvs = 0;  // one stream: PVs of earlier segments
    RingPos ring;  // of the segment's first load
    float x[COLS < 64 ? 64 : COLS];
    uint32_t joins = 0;  // phase of join[X]
    for (uint32_t tt = 0;; ++tt) {
      const int slot = tt % kInfoRing;
      if (!tree_wait(&ctl->info_full[slot], (tt / kInfoRing) & 1, abort, 6)) break;
      const Segment& sg = ctl->seg[slot];
      if (!sg.live) break;
      // the exchange of the last segment has been read by both streams
      if (tt > 0) {
        if (!tree_wait(&ctl->xchg_done, (tt - 1) & 1, abort, 7)) break;
        if (warp == 0 && lane < 2 * kTreeMaxWords) ctl->bad[(tt - 1) & 1][lane] = 0;
      }
      const int two = sg.two, nt = sg.nt, past = sg.past, n = sg.n;
      const int jt = (two ? X * p.tile_tokens : 0) + rj;  // the row's token within the unit
      const bool row_ok = rj < p.tile_tokens && jt < sg.ntok;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int t = sg.t0 + (row_ok ? jt : 0);
      const int j_seq = t - sg.seq_t0;  // its draft index
      int qpos = 0, lo_row = 0;
      float slope = 0.f;  // of the distance bias, in units of 1 / mul
      if constexpr (GEN) {
        qpos = p.positions ? p.positions[t] : past + j_seq;
        if (p.window >= 1) lo_row = max(max(qpos, past) - p.window + 1, 0);
        if (p.slopes && row_ok) slope = p.slopes[sg.k * p.G + (row - rj * p.G)] * (kLog2e / mul);
      }
      // Zero V rows that no row admits by position, take non-finite values out of
      // rows that only some admit: the drafts, and the context at the window's
      // edge (once per tile: stream 0 when both use it).  Unmapped pages and
      // pages behind the sequence are zero already.
      //
      // When: with GEN after the softmax, because a window's first V tiles come
      // later than their K (before it: a window of 1000 70.5 -> 72.2 us).  Else
      // before the wait for S, whose tensor work it then overlaps (head_size 64,
      // 128 sequences of 200..500 keys 46.2 -> 44.6 us, of 20..100 34.6 -> 33.6),
      // where that is sound.  The wait on the slot's parity means this load only
      // if the slot's load before it, n_v - S in the segment's order, has
      // landed.  It has if it belongs to an earlier segment.  Else: products
      // complete in order, so once S(i) is there so are loads 0 .. 2i - 1, and
      // n_v - S <= 2i - 1 for every S >= 3.  Before S(i) only the stream's tile
      // before i is known to be: with two row tiles loads 0 .. 2i - 2 (n_v =
      // 2i + 1; S >= 3), with the one stream of head_size 256 loads 0 .. 2i - 3
      // (n_v <= 2i + 2; S >= 5), with alternating tiles only 0 .. 2i - 5 (n_v <=
      // 2i + 2; S >= 7).  Alternating tiles of head_size 128 have 5 or 6 slots and
      // wait for S(i) (36.9 -> 37.1 us for units of one tile, nothing elsewhere).
      auto mend_v = [&](int i, int key0) -> bool {
        // no row admits a key below lo_min, and every row the context from lo_edge on
        const int lo_min = GEN && p.window >= 1 ? max(0, past + 1 - p.window) : 0;
        const int lo_edge = GEN && p.window >= 1 ? min(past - p.window + p.max_draft, past) : 0;
        // the tile's V load, counted from the segment's first, in the ring's order
        const int n_v = two ? 2 * i + 1 : (i == nt - 1 ? 2 * i + 1 : 2 * i + 2);
        const int turn = ring.slot + n_v, sv = turn % S;
        if constexpr (!GEN && !C::v_ordered(REP))
          if (!two && !tree_wait(&ctl->s_full[X], scnt & 1, abort, 16)) return false;
        if (!tree_wait(&ctl->full[sv], ring.phase ^ ((turn / S) & 1), abort, 10)) return false;
        uint8_t* vs = kv_s + sv * C::kSlotBytes;
        const int page_rows = 1 << log_r;
        const int k_lo = min(max(lo_min - key0, 0), kKeys);      // rows below: zero
        const int k_draft = min(max(past - key0, 0), kKeys);     // draft rows from here on
        const int k_edge = min(max(lo_edge - key0, 0), kKeys);   // (not above k_draft)
        const int k_end = min(max(past + n - key0, 0), kKeys);   // rows from here on: zero
        const int k_page = min((k_end + page_rows - 1) & ~(page_rows - 1), kKeys);  // ... up to here
        constexpr int kVecs = C::kChunks * 8;  // 16-byte vectors of a row
#pragma unroll 1
        for (int idx = r; idx < (k_edge + k_page - k_draft) * kVecs; idx += kRows) {
          int kr = idx / kVecs;
          const int v8 = idx % kVecs;
          if (kr >= k_edge) kr += k_draft - k_edge;
          uint4* at = reinterpret_cast<uint4*>(vs + (kr >> 3) * C::kGroupBytes + (v8 >> 3) * 1024 + (kr & 7) * 128 +
                                               (((v8 & 7) ^ (kr & 7)) << 4));
          if (kr < k_lo || kr >= k_end) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
          }
          const uint4 v = *at;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if (nonfinite_halves<BF>(w[0]) | nonfinite_halves<BF>(w[1]) | nonfinite_halves<BF>(w[2]) |
              nonfinite_halves<BF>(w[3])) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] &= ~((nonfinite_halves<BF>(w[e]) >> 15) * 0xffffu);
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            const int bit = key0 + kr - (kr >= k_draft ? past : lo_min - kTreeMaxDraft);
            atomicOr(&ctl->bad[tt & 1][bit >> 5], 1u << (bit & 31));
          }
        }
        fence_proxy_async_smem();
        return true;
      };
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      // a stream's tiles: all of them (two row tiles), every other one, or, as the one stream, all
      for (int i = C::kOneO ? X * nt : (two ? 0 : X); i < nt; i += C::kOneO || two ? 1 : 2) {
        const int buf = C::kOneO ? i & 1 : X;  // S and P columns
        const uint32_t tile = g + i;
        const int key0 = sg.key0 + i * kKeys;
        // (published before the tile's K load: read before the wait for S,
        // which hides the shared-memory load)
        if (!tree_wait(&ctl->mask_full[tile % kMaskRing], (tile / kMaskRing) & 1, abort, 8)) {
          ok = false;
          break;
        }
        const uint32_t pmask = ctl->kv_mask[tile % kMaskRing];
        // A tile that is not admitted as a whole: one bit per key of this row
        // (made before the wait for S).
        // (Lanes without a row compute on whatever Q's buffer holds there: no
        // other row sees it.)
        const bool partial = key0 + kKeys > past || pmask != 0 || __any_sync(0xffffffffu, row_ok && key0 < lo_row);
        const bool drafts = key0 + kKeys > past;
        constexpr int NW = COLS / 32;
        uint32_t w[NW];
        float ahead[NW];  // GEN: lane e, entry q: position of key cb + 32 q + e, less its slot
#pragma unroll
        for (int q = 0; q < NW; ++q) {
          w[q] = ~0u;
          ahead[q] = 0.f;
        }
        if (partial && warp_ok) {
          int kp[NW];
          if constexpr (GEN) {
            if (drafts && p.positions) {
#pragma unroll
              for (int q = 0; q < NW; ++q) {
                const int d = key0 + cb + 32 * q + lane - past;
                kp[q] = d >= 0 && d < n ? p.positions[sg.seq_t0 + d] : past + d;
                ahead[q] = (float)(kp[q] - (past + d));
              }
            }
          }
#pragma unroll
          for (int q = 0; q < NW; ++q) {
            const int k0 = key0 + cb + 32 * q, d0 = k0 - past;  // d0: draft index of bit 0
            uint32_t m = bit_range(lo_row - k0, -d0);
            if (d0 + 32 > 0 && d0 < n) {
              uint32_t md = bit_range(-d0, n - d0);
              if (p.mask) {
                const uint32_t* mrow = p.mask + (size_t)t * p.words;
                const int wi = d0 >> 5;  // (floor)
                const uint32_t a = wi >= 0 ? mrow[wi] : 0u;
                const uint32_t b = wi + 1 < p.words ? mrow[wi + 1] : 0u;
                md &= __funnelshift_r(a, b, d0 & 31);
              } else {
                md &= bit_range(0, j_seq + 1 - d0);
              }
              if constexpr (GEN) {
                if (p.window >= 1) {
                  uint32_t in = 0;
                  if (p.positions) {
                    // (as a rule no row's window leaves a draft token out)
                    const int d = d0 + lane, far = __reduce_min_sync(0xffffffffu, d >= 0 && d < n ? kp[q] : 0x7fffffff);
                    if (__any_sync(0xffffffffu, far < lo_row)) {
#pragma unroll 1
                      for (int e = 0; e < 32; ++e) in |= (__shfl_sync(0xffffffffu, kp[q], e) >= lo_row ? 1u : 0u) << e;
                    } else {
                      in = ~0u;
                    }
                  } else {
                    in = bit_range(lo_row - k0, 32);
                  }
                  md &= in;
                }
              }
              m |= md;
            }
            w[q] = row_ok ? m : 0u;
          }
          if (pmask != 0) {
#pragma unroll 1
            for (int g2 = 0; g2 < pages; ++g2) {
              if (!((pmask >> g2) & 1)) continue;
#pragma unroll
              for (int q = 0; q < NW; ++q)
                w[q] &= ~bit_range((g2 << log_r) - cb - 32 * q, ((g2 + 1) << log_r) - cb - 32 * q);
            }
          }
        }
        const bool mend = (drafts || (GEN && p.window >= 1 && key0 < past - p.window + p.max_draft)) && (!two || X == 0);
        if (!GEN && mend && !mend_v(i, key0)) {
          ok = false;
          break;
        }
        if (!tree_wait(&ctl->s_full[buf], (C::kOneO ? scnt >> buf : scnt) & 1, abort, 9)) {
          ok = false;
          break;
        }
        const bool first = i == (two || C::kOneO ? 0 : X);
        if constexpr (C::kOneO) scnt ^= 1u << buf;  // (a parity per buffer)
        else ++scnt;
        tc_fence_after();
        if (warp_ok) {
#pragma unroll
          for (int c = 0; c < COLS; c += 32) tmem_ld32(lane_addr + C::s_col(buf) + cb + c, x + c);
          tmem_ld_wait();
          if constexpr (GEN) {
            if (p.softcap > 0.f) {
              // x = tanh(y), y = S scale / c, in units of the cap c.  Where no |y| of
              // the warp is above 0.7 (scores well below the cap, the usual case)
              // by the polynomial y p(y^2) that meets tanh at the Chebyshev points
              // of y^2 in [0, 0.5] (off by 4.1e-7 relative), two columns per
              // instruction and no exponential unit; otherwise 1 - 2 / (1 + e^{2y}),
              // whose approximate reciprocal is off by 2^-23 of a term below 2.
              const float in = p.scale / p.softcap;
              float top = 0.f;
#pragma unroll
              for (int c = 0; c < COLS; c += 2) top = max3(top, fabsf(x[c]), fabsf(x[c + 1]));
              if (__any_sync(0xffffffffu, row_ok && !(top * fabsf(in) <= 0.7f))) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) x[c] = fmaf(-2.f, rcp(1.f + ex2(x[c] * (2.f * kLog2e * in))), 1.f);
              } else {
                const uint64_t in2 = f2(in, in);
#pragma unroll
                for (int c = 0; c < COLS; c += 2) {
                  const uint64_t y = mul2(f2(x[c], x[c + 1]), in2), t = mul2(y, y);
                  uint64_t a = f2(0.0136421223f, 0.0136421223f);
                  a = fma2(a, t, f2(-0.0507202948f, -0.0507202948f));
                  a = fma2(a, t, f2(0.132779678f, 0.132779678f));
                  a = fma2(a, t, f2(-0.333299451f, -0.333299451f));
                  a = fma2(a, t, f2(0.999999663f, 0.999999663f));
                  unf2(mul2(y, a), x[c], x[c + 1]);
                }
              }
            }
            // the bias's part that grows along the tile (`shift` holds the rest;
            // without a bias the slope is 0)
#pragma unroll
            for (int c = 0; c < COLS; ++c) x[c] = fmaf(slope, (float)c, x[c]);
          }
          if (partial) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
              // (draft tokens stand at positions of their own)
              const float moved = GEN ? fmaf(slope, __shfl_sync(0xffffffffu, ahead[c >> 5], c & 31), x[c]) : x[c];
              x[c] = ((w[c >> 5] >> (c & 31)) & 1) ? moved : -INFINITY;
            }
          }
          const float shift = GEN ? slope * (float)(key0 + cb - qpos) * mul : 0.f;
          const float cand = fmaf(max_tree<COLS>(x), mul, shift);
          float alpha = 1.f;
          if (cand > m_ref + kLazyRescale || (m_ref == -INFINITY && cand != -INFINITY)) {
            alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - cand);
            m_ref = cand;
          }
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t mul_2 = f2(mul, mul), neg_m2 = f2(shift - m_use, shift - m_use);
          uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int h = 0; h < COLS; h += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const uint64_t arg = fma2(f2(x[h + 2 * q], x[h + 2 * q + 1]), mul_2, neg_m2);
              float a0, a1;
              unf2(arg, a0, a1);
              const float e0 = ex2(a0), e1 = ex2(a1);
              sum2[q & 3] = add2(sum2[q & 3], f2(e0, e1));
              pk[q] = pack2<BF>(e0, e1);
            }
            // P -> TMEM over S: keys h..h+31 as 16 columns of 16-bit pairs
            tmem_st16(lane_addr + C::s_col(buf) + (cb + h) / 2, pk);
          }
          if constexpr (REP > 1) {  // ... and zeros at the other replicas' keys
            const uint32_t zero[16] = {};
#pragma unroll
            for (int h = 0; h < kKeys; h += 32)
              if (h < cb || h >= cb + COLS) tmem_st16(lane_addr + C::s_col(buf) + h / 2, zero);
          }
          if constexpr (C::kOneO) {
            // S(i) was issued before PV(i - 1): O is rescaled, and P(i) handed
            // over, only once that has completed.
            if (!first && !tree_wait(&ctl->pv_done, (pvs + i - 1) & 1, abort, 15)) {
              ok = false;
              break;
            }
            tc_fence_after();
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
        if (GEN && mend && !mend_v(i, key0)) {
          ok = false;
          break;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[buf]);
      }
      if (!ok) break;

      // ---- end of the segment: the streams show each other their maxima and
      // sums (needed when they hold the same rows), then O leaves TMEM.  A row
      // whose sum is no number (NaN or infinite scores) gets such a maximum,
      // whatever it met first: -inf means a row without keys, here and in the
      // joins, and fmaxf passes over a NaN.
      if (l != l) m_ref = l;
      ctl->ml[X][r] = make_float2(m_ref, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->xchg_full);
      if (!tree_wait(&ctl->xchg_full, tt & 1, abort, 11)) break;
      // Factors of O_0 and O_1 (one row tile), negative where the row met no
      // key (its O may be 0 * inf); a factor of 0 is applied, so that NaN and
      // infinities among the values are not lost.
      float f0 = 1.f, f1 = 1.f;
      if (!two) {
        // over both streams and all replicas of the row
        float2 ml[2 * REP];
        m_ref = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * REP; ++i) {
          ml[i] = ctl->ml[i & 1][(i >> 1) * R + row];
          m_ref = fmaxf(m_ref, ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < 2 * REP; ++i) {
          const float f = ml[i].x == -INFINITY ? -1.f : ex2(ml[i].x - m_ref);
          if (!(f < 0.f)) l += f * ml[i].y;
          if ((i >> 1) == (REP > 1 ? r / R : 0)) {
            if (i & 1) f1 = f;
            else f0 = f;
          }
        }
        if (l != l) m_ref = l;
      }
      uint32_t any_bad = lane < 2 * kTreeMaxWords ? ctl->bad[tt & 1][lane] : 0u;
      any_bad = __any_sync(0xffffffffu, any_bad != 0);
      const bool keep_bad = any_bad != 0;  // read again after the stores: released there
      if (lane == 0 && !keep_bad) mbar_arrive(&ctl->xchg_done);
      const int jobs = two ? 2 * nt : nt;
      bool have[2] = {true, !C::kOneO && jobs >= 2};
      for (int Y = 0; Y < 2 && ok; ++Y) {
        if (!have[Y]) continue;
        if ((!two || Y == X) &&
            !tree_wait(&ctl->o_done[Y], ocnt[Y] & 1, abort, 13))
          ok = false;
        ++ocnt[Y];
      }
      if (!ok) break;
      tc_fence_after();
      const int h = sg.k * p.G + (row - rj * p.G);
      float inv = 1.f;
      if (sg.slot < 0) {
        if (p.head_sink && row_ok && m_ref != -INFINITY)
          l += ex2(elem16_to_float(p.head_sink[h], BF) * kLog2e - m_ref);
        inv = l == 0.f ? 0.f : 1.f / l;
      }
      const int urow = (two ? X * kRows : 0) + row;  // row of the unit's partial result
      if (sg.slot >= 0 && row_ok && (two || threadIdx.x < R))
        p.part_ml[(size_t)sg.slot * p.part_rows + urow] = make_float2(m_ref, l);
      __half* dst = p.out + ((size_t)t * p.H + h) * D;
      float4* part = sg.slot >= 0 ? p.part_o + (size_t)sg.slot * (D / 4) * p.part_rows + urow : nullptr;
      // Two row tiles: every channel of the own O; one: half the channels of both.
      const int c0 = two ? 0 : X * (D / 2), c1 = two ? D : c0 + D / 2;
      if constexpr (REP > 1) {
        // The replicas' O, scaled, side by side in shared memory, 16 channels
        // of this stream's half at a time; then each thread adds up four
        // channels of a row in replica order and stores them.
        float4* red = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(ctl) + kCtrlBytes) + X * kRows * kJoinChannels / 4;
        float2* stat = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(ctl) + kCtrlBytes + 2 * kRows * kJoinChannels * 4) +
                       X * kRows;
        auto join_all = [&]() -> bool {  // the four warps of this stream
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->join[X]);
          return tree_wait(&ctl->join[X], joins++ & 1, abort, 14);
        };
        if (r < R) stat[row] = make_float2(__int_as_float(row_ok ? t * p.H + h : -1), l == l ? inv : l);
#pragma unroll 1
        for (int c = c0; c < c1 && ok; c += kJoinChannels) {
          if (warp_ok) {
            tmem_ld16(lane_addr + C::o_col(0) + c, x);
            if (have[1]) tmem_ld16(lane_addr + C::o_col(1) + c, x + 16);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              x[e] = f0 < 0.f ? 0.f : x[e] * f0;
              if (!(f1 < 0.f)) x[e] = fmaf(x[16 + e], f1, x[e]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)  // (the exchange of vectors spreads a warp's stores over the banks)
              red[r * 4 + (q ^ ((r >> 1) & 3))] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          }
          ok = join_all();
#pragma unroll
          for (int i = 0; i < R * 4 / kRows && ok; ++i) {
            const int item = i * kRows + r, orow = item >> 2, q = item & 3;
            const float2 st = stat[orow];
            const int at = __float_as_int(st.x);  // (token, head) of the row, -1: none
            if (at < 0) continue;
            float4 v = red[orow * 4 + (q ^ ((orow >> 1) & 3))];
#pragma unroll
            for (int k = 1; k < REP; ++k) {
              const float4 u = red[(k * R + orow) * 4 + (q ^ ((orow >> 1) & 3))];
              v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            const float sum = (v.x + v.y) + (v.z + v.w);
            if (sum != sum && st.y == st.y) ctl->lost[X] = 1;  // (every writer stores the same value)
            if (sg.slot >= 0)
              p.part_o[((size_t)sg.slot * (D / 4) + c / 4 + q) * p.part_rows + orow] = v;
            else
              *reinterpret_cast<uint2*>(p.out + (size_t)at * D + c + 4 * q) =
                  make_uint2(pack2<BF>(v.x * st.y, v.y * st.y), pack2<BF>(v.z * st.y, v.w * st.y));
          }
          ok = ok && join_all();
        }
        if (!ok) break;
        if (*static_cast<volatile uint32_t*>(&ctl->lost[X])) {
          // A replica's P is 0 at the others' keys, and 0 * inf is NaN: an
          // infinity in a context key was lost.  Which of the stream's channels
          // hold one (or a NaN, or both signs) is read off the keys that every
          // row admits and nobody has mended, and put in place of the NaN.
          static_assert(D / 2 == 32, "a channel per bit");
          const int first = GEN && p.window >= 1 ? max(sg.key0, min(past - p.window + p.max_draft, past)) : sg.key0;
          const int last = min(past, sg.key0 + nt * kKeys);
          uint32_t up = 0, down = 0, none = 0;  // +inf, -inf, NaN
#pragma unroll 1
          for (int pos = first + r; pos < last; pos += kRows) {
            const int blk = p.block_table[(size_t)sg.b * p.MB + (pos >> p.log_bs)];
            if (blk < 0 || blk >= p.NB) continue;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(
                p.value_cache + ((((size_t)blk << p.log_bs) + (pos & (p.bs - 1))) * p.Hk + sg.k) * D + c0);
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
              const uint32_t two_halves = v[i];
              if (!nonfinite_halves<BF>(two_halves)) continue;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t half = two_halves >> (16 * e) & 0xffffu;
                if (!nonfinite16<BF>(half)) continue;
                const uint32_t bit = 1u << (2 * i + e);
                if (half & (BF ? 0x7fu : 0x3ffu)) none |= bit;
                else if (half >> 15) down |= bit;
                else up |= bit;
              }
            }
          }
          if (up) atomicOr(&ctl->found[X][0], up);
          if (down) atomicOr(&ctl->found[X][1], down);
          if (none) atomicOr(&ctl->found[X][2], none);
          if (!(ok = join_all())) break;
          const volatile uint32_t* found = ctl->found[X];
          up = found[0];
          down = found[1];
          none = (up & down) | found[2];
          if (row_ok && r < R && l == l) {
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
              const uint32_t bit = 1u << (c - c0);
              if (!((up | down) & ~none & bit)) continue;
              const float value = up & bit ? INFINITY : -INFINITY;
              float* po = part ? reinterpret_cast<float*>(part + (size_t)(c / 4) * p.part_rows) + (c & 3) : nullptr;
              const float was = part ? *po : elem16_to_float(dst[c], BF);
              if (was == was) continue;
              if (part) *po = value;
              else dst[c] = float_to_elem16(value, BF);
            }
          }
          if (!(ok = join_all())) break;
          if (r < 3) ctl->found[X][r] = 0;
          if (r == 3) ctl->lost[X] = 0;
        }
      } else if (warp_ok) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          tmem_ld32(lane_addr + C::o_col(0) + (two ? X * D : 0) + c, x);
          if (have[1] && !two) tmem_ld32(lane_addr + C::o_col(1) + c, x + 32);
          tmem_ld_wait();
          if (!two) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              x[e] = f0 < 0.f ? 0.f : x[e] * f0;
              if (!(f1 < 0.f)) x[e] = fmaf(x[32 + e], f1, x[e]);
            }
          }
          if (row_ok) {
            if (part) {
              float4* at = part + (size_t)(c / 4) * p.part_rows;
#pragma unroll
              for (int q = 0; q < 8; ++q, at += p.part_rows) *at = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(dst + c + 8 * q) =
                    make_uint4(pack2<BF>(x[8 * q] * inv, x[8 * q + 1] * inv), pack2<BF>(x[8 * q + 2] * inv, x[8 * q + 3] * inv),
                               pack2<BF>(x[8 * q + 4] * inv, x[8 * q + 5] * inv),
                               pack2<BF>(x[8 * q + 6] * inv, x[8 * q + 7] * inv));
            }
          }
        }
      }
      // O may be overwritten by the next segment's first PV
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->o_free[0]);
        mbar_arrive(&ctl->o_free[1]);
      }
      if (any_bad && row_ok && r < R) {
        // Keys with non-finite V: added, element by element, to what has just
        // been stored for the row if the row admits them.
#pragma unroll 1
        for (int i = 0; i < 2 * kTreeMaxDraft; ++i) {
          const uint32_t left = ctl->bad[tt & 1][i >> 5] >> (i & 31);
          if (left == 0) i |= 31;
          if (!(left & 1)) continue;
          const bool draft = i < kTreeMaxDraft;
          if (draft && !mask_bit(p, t, j_seq, i)) continue;
          const int pos = draft ? past + i : max(0, past + 1 - p.window) + i - kTreeMaxDraft;
          if (GEN && p.window >= 1 && (draft && p.positions ? p.positions[sg.seq_t0 + i] : pos) < lo_row) continue;
          const int blk = p.block_table[(size_t)sg.b * p.MB + (pos >> p.log_bs)];
          if (blk < 0 || blk >= p.NB) continue;
          const __half* v =
              p.value_cache + ((((size_t)blk << p.log_bs) + (pos & (p.bs - 1))) * p.Hk + sg.k) * D;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            if (!nonfinite16<BF>(__half_as_ushort(v[c]))) continue;
            const float add = elem16_to_float(v[c], BF);
            if (part) reinterpret_cast<float*>(part + (size_t)(c / 4) * p.part_rows)[c & 3] += add;
            else dst[c] = float_to_elem16(elem16_to_float(dst[c], BF) + add, BF);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && keep_bad) mbar_arrive(&ctl->xchg_done);
      const int turn = ring.slot + 2 * nt;
      ring.phase ^= (turn / S) & 1;
      ring.slot = turn % S;
      pvs += nt;
      if (lane == 0) mbar_arrive(&ctl->info_empty[slot]);
      g += nt;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) note_timeout(p.err, p.err_site, *abort);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the partial results of the units that range borders cut; a warp takes
// 8 channels of some rows.  Units in two pieces (the front of the list of
// cuts): 32 rows at a time, a lane is a row and loads both at once.  Units in
// more pieces (the back of the list): 8 rows at a time times four shares of
// the pieces (every fourth one), added by shuffles.  Partials are stored
// channel group by channel group with rows side by side, so both kernels
// access whole sectors.  The last block to finish clears the counters.
// Bound by L2: about 8 us for the 47 MB of 144 units of 256 rows of 128
// channels, of which 3 us are the launch.  (In the main kernel, by whoever
// writes a unit's last piece: 158 us against 145 at two long sequences.)
template <int D, bool BF>
__global__ void __launch_bounds__(D / 8 * 32) tree_join_kernel(const __grid_constant__ TreeParams p) {
  const int lane = threadIdx.x & 31, c8 = threadIdx.x >> 5;
  const int groups2 = p.part_rows / 32, groups = p.part_rows / 8;
  griddep_wait();
  griddep_launch_dependents();
  const int n2 = p.counters->n_cuts[0] * groups2, n_work = n2 + p.counters->n_cuts[1] * groups;
  const int last = p.n_ranges * p.Hk - 1;  // of the list
  Cut cut{};
  // out = acc / (den + sink) of one row
  auto store = [&](int row, float m, float den, const float* acc) {
    const int X = row / kRows, r = row - X * kRows, rj = r / p.G, j = X * p.tile_tokens + rj;
    if (row >= cut.rows || rj >= p.tile_tokens || j >= cut.ntok) return;
    const int t = cut.t0 + j, h = cut.k * p.G + (r - rj * p.G);
    if (p.head_sink && m != -INFINITY) den += ex2(elem16_to_float(p.head_sink[h], BF) * kLog2e - m);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    *reinterpret_cast<uint4*>(p.out + ((size_t)t * p.H + h) * D + 8 * c8) =
        make_uint4(pack2<BF>(acc[0] * inv, acc[1] * inv), pack2<BF>(acc[2] * inv, acc[3] * inv),
                   pack2<BF>(acc[4] * inv, acc[5] * inv), pack2<BF>(acc[6] * inv, acc[7] * inv));
  };
  for (int i = blockIdx.x; i < n_work; i += gridDim.x) {
    if (i < n2) {
      cut = p.cuts[i / groups2];
      const int row = i % groups2 * 32 + lane;
      if (row - lane >= cut.rows) continue;
      const size_t at0 = cut.slot0, at1 = cut.slot1;
      const float4* o0 = p.part_o + (at0 * (D / 4) + 2 * c8) * p.part_rows + row;
      const float4* o1 = p.part_o + (at1 * (D / 4) + 2 * c8) * p.part_rows + row;
      const float2 ml0 = p.part_ml[at0 * p.part_rows + row], ml1 = p.part_ml[at1 * p.part_rows + row];
      const float4 a0 = o0[0], b0 = o0[p.part_rows], a1 = o1[0], b1 = o1[p.part_rows];
      const float m = fmaxf(ml0.x, ml1.x);
      // (negative: no key)
      const float f0 = ml0.x == -INFINITY ? -1.f : ex2(ml0.x - m), f1 = ml1.x == -INFINITY ? -1.f : ex2(ml1.x - m);
      const float v0[8] = {a0.x, a0.y, a0.z, a0.w, b0.x, b0.y, b0.z, b0.w};
      const float v1[8] = {a1.x, a1.y, a1.z, a1.w, b1.x, b1.y, b1.z, b1.w};
      float acc[8], den = f0 < 0.f ? 0.f : f0 * ml0.y;
      if (!(f1 < 0.f)) den += f1 * ml1.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[e] = f0 < 0.f ? 0.f : f0 * v0[e];
        if (!(f1 < 0.f)) acc[e] += f1 * v1[e];
      }
      store(row, m, den, acc);
    } else {
      cut = p.cuts[last - (i - n2) / groups];
      const int row = (i - n2) % groups * 8 + (lane & 7), ns = cut.more + 1;
      if (row - (lane & 7) >= cut.rows) continue;
      auto slot_of = [&](int s) -> size_t { return s == 0 ? cut.slot0 : cut.slot1 + 2 * p.Hk * (s - 1); };
      float m = -INFINITY, den = 0.f, acc[8] = {};
#pragma unroll 2
      for (int s = lane >> 3; s < ns; s += 4) {
        const size_t at = slot_of(s);
        const float2 ml = p.part_ml[at * p.part_rows + row];
        const float4* o = p.part_o + (at * (D / 4) + 2 * c8) * p.part_rows + row;
        const float4 a = o[0], b = o[p.part_rows];
        if (ml.x == -INFINITY) continue;
        const float m_new = fmaxf(m, ml.x), f_old = m == -INFINITY ? 0.f : ex2(m - m_new), f = ex2(ml.x - m_new);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        den = den * f_old + ml.y * f;  // (a NaN stays one)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = acc[e] * f_old + v[e] * f;
        m = m_new;
      }
      float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
      const float f = m == -INFINITY ? 0.f : ex2(m - M);
      den *= f;  // (0 without keys)
      den += __shfl_xor_sync(0xffffffffu, den, 8);
      den += __shfl_xor_sync(0xffffffffu, den, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[e] *= f;
        acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], 8);
        acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], 16);
      }
      if (lane < 8) store(row, M, den, acc);
    }
  }
  __syncthreads();  // every warp has read n_cuts
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&p.counters->joined, 1) == (int)gridDim.x - 1) {
      p.counters->n_cuts[0] = 0;
      p.counters->n_cuts[1] = 0;
      p.counters->joined = 0;
    }
  }
}

template <int D, bool BF, bool GEN, int REP>
cudaError_t configure() {
  using C = TreeCfg<D>;
  static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");
  constexpr int kQTiles = REP > 1 || C::kOneO ? 1 : 2;
  static_assert(C::smem_bytes(1, REP) <= kSmemLimit && C::smem_bytes(kQTiles, REP) <= kSmemLimit, "shared memory");
  static_assert(C::slots(kQTiles, REP) >= 4 && kMaxSlots / 2 + 3 <= kMaskRing, "K/V ring");
  static_assert(2 * C::kKeys + (C::kOneO ? 1 : 2) * D <= C::kTmemCols, "tensor memory");
  static_assert(C::v_ordered(REP) || (!C::kOneO && C::slots(kQTiles, REP) >= 3), "V slots waited for in order");
  return cudaFuncSetAttribute(tree_kernel<D, BF, GEN, REP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              std::max(C::smem_bytes(1, REP), C::smem_bytes(kQTiles, REP)));
}

template <int D, bool BF, int REP>
cudaError_t configure_dbr() {
  const cudaError_t e = configure<D, BF, false, REP>();
  return e != cudaSuccess ? e : configure<D, BF, true, REP>();
}

template <int D, bool BF, int REP>
cudaError_t launch_dbr(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                       int grid, cudaStream_t s) {
  const bool gen = p.softcap > 0.f || p.slopes || p.window >= 1;
  const int smem = TreeCfg<D>::smem_bytes(p.q_tiles, REP);
  cudaError_t e = gen ? launch_pdl(tree_kernel<D, BF, true, REP>, dim3(grid), kThreads, smem, s, tq, tk, tv, p)
                      : launch_pdl(tree_kernel<D, BF, false, REP>, dim3(grid), kThreads, smem, s, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_join_kernel<D, BF>, dim3(2 * grid), D / 8 * 32, 0, s, p);
}

// One translation unit per head size (PA_TREE_D), so that they compile side by side.
template <bool BF>
cudaError_t configure_bf(int rep) {
#if PA_TREE_D == 64
  if (rep == 4) return configure_dbr<64, BF, 4>();
  if (rep == 2) return configure_dbr<64, BF, 2>();
#endif
  return configure_dbr<PA_TREE_D, BF, 1>();
}

template <bool BF>
cudaError_t launch_bf(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, int grid,
                      cudaStream_t s) {
#if PA_TREE_D == 64
  if (p.rep == 4) return launch_dbr<64, BF, 4>(tq, tk, tv, p, grid, s);
  if (p.rep == 2) return launch_dbr<64, BF, 2>(tq, tk, tv, p, grid, s);
#endif
  return launch_dbr<PA_TREE_D, BF, 1>(tq, tk, tv, p, grid, s);
}

}  // namespace

template <>
cudaError_t tree_configure<PA_TREE_D>(int bf16, int rep) {
  return bf16 ? configure_bf<true>(rep) : configure_bf<false>(rep);
}

template <>
cudaError_t launch_tree<PA_TREE_D>(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const TreeParams& p, int bf16, int grid, cudaStream_t s) {
  return bf16 ? launch_bf<true>(tq, tk, tv, p, grid, s) : launch_bf<false>(tq, tk, tv, p, grid, s);
}

}  // namespace pa
