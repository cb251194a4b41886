// Attention over pools held in 4 bits for sequences with many query rows
// (chunks of prompts, long drafts), on tcgen05 (head_size 64 and 128).
//
// S = Q K^T and O += P V with 128-row tiles in tensor memory.  The operands
// K and V are made from the codes: a warpgroup takes a key per thread, turns
// its codes into (n - 8) / 8 (two exact fp16 operations: an or that puts the
// nibble behind a power of two, a subtraction) and multiplies by the group's
// scale, which rounds the value to fp16 once, and stores the row where a
// 128-byte-swizzled tile has it.  The 1/8 keeps 8 times the largest scale in
// fp16's range; f and the output take it back.  A query row is brought near
// the top of fp16's range by a power of two, so that nothing of it is lost,
// whatever the activations' type.
//
// Work.  A unit is up to 256 rows (token x head) of a sequence and kv head,
// tiles A and B of 128; every 128-key tile of K and V made is used by both,
// and while one tile's softmax runs the tensor core multiplies for the
// other.  The key tiles of all units stand in one line, cut into one equal
// range per SM; a unit that a border cuts leaves partial results that a
// last kernel joins.
//
// A unit of at most 128 rows has no tile B; both softmax warpgroups then take
// the one tile's rows, over every other key tile each, with sums and outputs
// of their own that A joins at the end.  Otherwise scores, softmax and product
// of one key tile after the other wait for each other: 32 sequences of 36 rows
// after 3,000 tokens, 8 kv heads of 128, take 158 us without and 134 with it.
// Calls with more than 128 rows to a sequence get a kernel without this part:
// it costs them 2 % to 8 % (the chunks below: 577 us became 586).
//
// What bounds it.  Two chunks of 1,024 tokens after 8,000 to 16,000, 32 query
// heads over 8 of 128: 575 us, where the products alone are 252 us at the
// bf16 rate that a library product reaches.  The tensor cores are busy 36 % of
// the time, instructions issue 44 %: each tile's scores, softmax, P and
// product follow one another, and at head_size 128 two tiles' S and O fill
// tensor memory, so there is no third to fill the gaps.  The roles' code
// together is about what the instruction caches hold (fetch at 70 % of its
// peak), hence the loops below that could be unrolled.
//
// Roundings beyond the scores' and sums' 32 bits: an eighth of a K or V value to
// fp16 (a code times its scale has up to 14 bits; values below 2^-11 go to
// multiples of 2^-21), a weight to fp16.  The outputs of those chunks are
// 4.9e-4 off (relative, root mean square), 2.1e-4 of it their own rounding to
// fp16.
//
// Roles (640 threads, one CTA per SM; registers moved between warpgroups):
//   warpgroups 0, 1: tile A, B: the query's operand, softmax, output
//     (thread = row = tensor memory lane);
//   warpgroups 2, 3: the operand K, V (thread = key);
//   warpgroup 4: warp 16 finds the units, warp 17 issues the MMAs.
#include <algorithm>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "q4.h"
#include "step.h"

namespace pa {
namespace {

constexpr int kThreads = 640;
constexpr int kMakeWarp0 = 8, kFetchWarp = 16, kMmaWarp = 17;
// Registers per thread after the split (launch: 96 each; the warpgroups that
// make operands keep theirs).
constexpr int kRegSoftmax = 120, kRegControl = 48;
static_assert(2 * kRegSoftmax + 2 * 96 + kRegControl <= 5 * 96, "register split");
constexpr int kTile = 128;         // rows of a tile, keys of a tile
constexpr int kInfoRing = 4;
constexpr int kMaskRing = 8;       // tiles whose masks are held: more than the ring of operands runs ahead
constexpr int kSmemLimit = 227 * 1024;
constexpr int kCtrlBytes = 2048;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are exp2(score - reference), the reference a whole number: it starts
// kLift below the largest score and moves when one passes it by kLift +
// kSlack.  The largest weight then lies between 2^5 and 2^14 of fp16's 2^16,
// and one 2^-19 as large still keeps all of its bits (with a reference at
// the largest score, 8,192 keys of 2^-25.4 each were lost, 2e-4 of a row); and
// what a move multiplies by is a power of two, which rounds no weight a second
// time unless it falls below fp16's smallest normal.
constexpr float kLift = 6.f, kSlack = 8.f;
constexpr int kSite = kSiteQ4 | 64;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;  // [chunk][row][128 B]
  static constexpr int kFit = (kSmemLimit - 1024 - kCtrlBytes - 2 * kTileBytes) / kTileBytes;
  static constexpr int kSlots = kFit > 6 ? 6 : kFit;  // K_i is load 2i, V_i load 2i + 1
  static constexpr int kSmem = 1024 + (2 + kSlots) * kTileBytes + kCtrlBytes;
  static __host__ __device__ constexpr int s_col(int X) { return X * kTile; }
  static __host__ __device__ constexpr int o_col(int X) { return 2 * kTile + X * D; }
  static constexpr int kTmemCols = 512;
};

struct Unit {
  int n;            // key tiles of it in this range; 0: no more units
  int i0;           // the first of them
  int first_tiles, lo;  // tiles below the window, and the position at which the others start
  int h, b, t0;     // kv head, sequence, packed row of its first token
  int row0, nrows;  // rows of the (sequence, kv head)
  int past, pos_max, lo_min;  // of its rows: largest position, smallest that a window admits
  int part;         // slot of its partial results, -1: the whole unit is here
  int pad[3];
};

// Whether both softmax warpgroups share the unit's one tile of rows.
__device__ __forceinline__ bool shared_tile(const Unit& u) { return u.nrows <= kTile && u.n > 1; }

struct TileMask {
  uint32_t unmapped[4], bad[4];  // per 32 keys: no page; a scale of V that is no number
};

struct Ctrl {
  Unit info[kInfoRing];
  TileMask mask[kMaskRing];
  uint64_t mask_full[kMaskRing];
  uint64_t info_full[kInfoRing], info_empty[kInfoRing];
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
  uint64_t b_ready, b_taken;  // B's sums of a shared tile are there; they and its output have been read
  uint64_t full[6], empty[6];
  uint64_t drain;
  long long scan[kThreads / 32];
  long long start_line;
  int start_seq;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

// Key tiles of row block u of a sequence.
struct Block {
  int first_tiles, lo, tiles, nrows;
};
__device__ __forceinline__ Block row_block(const Q4Params& p, int n, int past, int u) {
  Block k;
  const long long row0 = (long long)u * kQ4TileRows, rows = (long long)n * p.G - row0;
  k.nrows = (int)min((long long)kQ4TileRows, rows);
  const int pos_min = past + (int)(row0 / p.G), pos_max = past + (int)((row0 + k.nrows - 1) / p.G);
  k.lo = p.window > 0 ? max(0, pos_min + 1 - p.window) & ~(kTile - 1) : 0;
  k.first_tiles = (min(p.first, k.lo) + kTile - 1) / kTile;
  k.tiles = k.first_tiles + (pos_max + 1 - k.lo + kTile - 1) / kTile;
  return k;
}
__device__ __forceinline__ int tile_key(const Unit& u, int i) {
  return i < u.first_tiles ? kTile * i : u.lo + kTile * (i - u.first_tiles);
}

// Row blocks of sequence b that this kernel serves (0: none); flags bad lengths.
__device__ __forceinline__ int blocks_of(const Q4Params& p, int b, int* n, int* past) {
  const int c0 = p.g.cum[b], c1 = p.g.cum[b + 1];
  *past = p.g.past[b];
  *n = c1 - c0;
  // (the other kernel flags what is wrong)
  if (c0 < 0 || c1 <= c0 || c1 > p.g.T || *past < 0 || (long long)*past + *n > p.g.max_kv) return 0;
  if ((long long)*n * p.G <= p.stream_rows) return 0;
  return (int)(((long long)*n * p.G + kQ4TileRows - 1) / kQ4TileRows);
}


// Eight codes as (n - 8) / 8 times s (the same in both halves): channels in
// order.  Nibbles 0 and 2 of a half go behind 128 (unit 1/8), 1 and 3, which
// lie four bits higher, behind 8.
__device__ __forceinline__ uint4 make_values(uint32_t w, uint32_t s) {
  const uint32_t w8 = w >> 8;
  const uint32_t k129 = 0x58085808u, k9 = 0x48804880u;  // 129 and 9
  uint4 y;
  y.x = hmul2_bits(hsub2_bits((w & 0x000F000Fu) | 0x58005800u, k129), s);
  y.y = hmul2_bits(hsub2_bits((w & 0x00F000F0u) | 0x48004800u, k9), s);
  y.z = hmul2_bits(hsub2_bits((w8 & 0x000F000Fu) | 0x58005800u, k129), s);
  y.w = hmul2_bits(hsub2_bits((w8 & 0x00F000F0u) | 0x48004800u, k9), s);
  return y;
}

template <int D, bool CAP, bool SHARE>
__global__ void __launch_bounds__(kThreads, 1) q4_tile_kernel(const __grid_constant__ Q4Params p) {
  using C = Cfg<D>;
  constexpr int S = C::kSlots, kGroups = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                      // tiles A, B
  uint8_t* kv_s = smem + 2 * C::kTileBytes;
  Ctrl* ctl = reinterpret_cast<Ctrl*>(smem + (2 + S) * C::kTileBytes);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 4);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->o_done[i], 1);
    }
    for (int i = 0; i < kInfoRing; ++i) {
      mbar_init(&ctl->info_full[i], 1);
      mbar_init(&ctl->info_empty[i], 1 + 8 + 8);  // MMA, softmax and operand warps
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(&ctl->full[i], 4);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ctl->mask_full[i], 8);
    mbar_init(&ctl->b_ready, 4);
    mbar_init(&ctl->b_taken, 4);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ctl->start_seq = 0x7fffffff;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();

  // The line of key tiles: a warp sums a share of the sequences, 32 at a
  // time, and the one whose share holds the start of this CTA's range finds
  // the sequence.
  const int per = (p.g.batch + kThreads / 32 - 1) / (kThreads / 32), s0 = min(p.g.batch, warp * per), s1 = min(p.g.batch, s0 + per);
  auto each_seq = [&](auto visit) {  // visit(b, tiles x heads) until it says so
    for (int b0 = s0; b0 < s1; b0 += 32) {
      int n = 0, past = 0, blocks = 0;
      if (b0 + lane < s1) blocks = blocks_of(p, b0 + lane, &n, &past);
      for (unsigned has = __ballot_sync(0xffffffffu, blocks > 0); has; has &= has - 1) {
        const int src = __ffs(has) - 1;
        const int bn = __shfl_sync(0xffffffffu, n, src), bp = __shfl_sync(0xffffffffu, past, src);
        const int bb = __shfl_sync(0xffffffffu, blocks, src);
        long long len = 0;
        for (int u = lane; u < bb; u += 32) len += row_block(p, bn, bp, u).tiles;
#pragma unroll
        for (int d = 16; d; d >>= 1) len += __shfl_xor_sync(0xffffffffu, len, d);
        if (visit(b0 + src, len * p.g.Hk)) return;
      }
    }
  };
  long long sum = 0;
  each_seq([&](int, long long len) {
    sum += len;
    return false;
  });
  if (lane == 0) ctl->scan[warp] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long s = ctl->scan[w];
    if (w < warp) before += s;
    total += s;
  }
  const long long ranges = min((long long)gridDim.x, total), me = min((long long)blockIdx.x, ranges);
  const long long r0 = ranges ? total * me / ranges : 0, r1 = me < ranges ? total * (me + 1) / ranges : r0;
  if (r0 < r1 && r0 >= before && r0 < before + sum) {
    long long at = before;
    each_seq([&](int b, long long len) {
      if (r0 < at + len) {
        if (lane == 0) {
          ctl->start_seq = b;
          ctl->start_line = at;
        }
        return true;
      }
      at += len;
      return false;
    });
  }
  __syncthreads();

  if (warp >= kFetchWarp) {
   regs_dec<kRegControl>();
   if (warp == kFetchWarp) {
    // ------------------------------------------------------------- fetcher
    Q4Cut cut;
    cut.pieces = 0;
    long long x = r0, line = ctl->start_line;
    uint32_t n_units = 0;
    bool ok = true;
    for (int b = ctl->start_seq; ok && x < r1 && b < p.g.batch; ++b) {
      int n, past;
      const int blocks = blocks_of(p, b, &n, &past);
      const int t0 = blocks ? p.g.cum[b] : 0;
      for (int u = 0; ok && x < r1 && u < blocks;) {
        // the block that holds x, 32 at a time
        const long long mine = u + lane < blocks ? (long long)row_block(p, n, past, u + lane).tiles * p.g.Hk : 0;
        long long incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += y;
        }
        const unsigned behind = __ballot_sync(0xffffffffu, line + incl > x);
        if (!behind) {
          line += __shfl_sync(0xffffffffu, incl, 31);
          u += 32;
          continue;
        }
        const int at = __ffs(behind) - 1;
        line += __shfl_sync(0xffffffffu, incl - mine, at);
        u += at;
        const Block k = row_block(p, n, past, u);
        const long long len = (long long)k.tiles * p.g.Hk;
        while (ok && x < r1 && x < line + len) {
          const long long in = x - line;
          const int h = (int)(in / k.tiles), i0 = (int)(in - (long long)h * k.tiles);
          const int m = (int)min((long long)(k.tiles - i0), r1 - x);
          const bool from_start = i0 == 0, to_end = i0 + m == k.tiles;
          const uint32_t s = n_units % kInfoRing;
          int good = 1;
          if (lane == 0) {
            good = wait_or_abort(&ctl->info_empty[s], ((n_units / kInfoRing) & 1) ^ 1, abort, p.g.err, p.err_site, kSite | 1);
            if (good) {
              Unit& f = ctl->info[s];
              f.n = m;
              f.i0 = i0;
              f.first_tiles = k.first_tiles;
              f.lo = k.lo;
              f.h = h;
              f.b = b;
              f.t0 = t0;
              f.row0 = u * kQ4TileRows;
              f.nrows = k.nrows;
              f.past = past;
              f.pos_max = past + (f.row0 + k.nrows - 1) / p.G;
              f.lo_min = p.window > 0 ? max(0, past + f.row0 / p.G + 1 - p.window) : 0;
              f.part = from_start && to_end ? -1 : 2 * (int)blockIdx.x + (from_start ? 1 : 0);
              mbar_arrive(&ctl->info_full[s]);
            }
          }
          ok = __shfl_sync(0xffffffffu, good, 0);
          ++n_units;
          if (from_start && !to_end) {
            const long long last = x + k.tiles - 1;  // of the unit; the range that holds it
            cut.pieces = (int)(((last + 1) * ranges - 1) / total) - (int)blockIdx.x + 1;
            cut.t0 = t0;
            cut.row0 = u * kQ4TileRows;
            cut.nrows = k.nrows;
            cut.h = h;
          }
          x += m;
        }
        line += len;
        ++u;
      }
    }
    if (lane == 0) {
      p.tile_cuts[blockIdx.x] = cut;
      const uint32_t s = n_units % kInfoRing;
      if (ok && wait_or_abort(&ctl->info_empty[s], ((n_units / kInfoRing) & 1) ^ 1, abort, p.g.err, p.err_site, kSite | 1)) {
        ctl->info[s].n = 0;
        mbar_arrive(&ctl->info_full[s]);
      }
    }
   } else if (warp == kMmaWarp) {
    // --------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = umma_idesc_f16(kTile, kTile, 0, 0, 0);
    constexpr uint32_t idesc_o = umma_idesc_f16(kTile, D, 0, 1, 0);
    const uint64_t desc_k = smem_desc_sw128(0, 16, 1024);           // K-major Q and K, + (address >> 4)
    const uint64_t desc_v = smem_desc_sw128(0, kTile * 128, 1024);  // MN-major V, + (address >> 4)
    const uint32_t kv_addr = smem_u32(kv_s), q_addr = smem_u32(q_s);
    const bool leader = elect_one();
    auto wait_bar = [&](uint64_t* bar, uint32_t parity) -> bool {
      return wait_or_abort(bar, parity, abort, p.g.err, p.err_site, kSite | 2);
    };
    uint32_t g = 0, pcnt[2] = {0, 0}, qcnt[2] = {0, 0};
    bool ok = leader;
    for (uint32_t tt = 0; ok; ++tt) {
      const int slot = tt % kInfoRing;
      if (!wait_bar(&ctl->info_full[slot], (tt / kInfoRing) & 1)) break;
      const int n = ctl->info[slot].n, last_x = ctl->info[slot].nrows > kTile ? 1 : 0;
      if (n == 0) break;
      const bool share = SHARE && shared_tile(ctl->info[slot]);
      // S_X = Q_X K_i^T; the K tile is waited for by its first use and released
      // by its last.
      auto issue_s = [&](int X, int i, bool begins, bool first, bool last) -> bool {
        const uint32_t m = 2 * (g + i);
        const int st = m % S;
        if (begins) {
          if (!wait_bar(&ctl->q_full[X], qcnt[X] & 1)) return false;
          ++qcnt[X];
        }
        if (first && !wait_bar(&ctl->full[st], (m / S) & 1)) return false;
        tc_fence_after();
        const uint64_t a0 = desc_k + ((q_addr + X * C::kTileBytes) >> 4);
        const uint64_t b0 = desc_k + ((kv_addr + st * C::kTileBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_f16(tmem + C::s_col(X), a0 + (((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4),
                   b0 + (((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
        umma_commit(&ctl->s_full[X]);
        if (last) umma_commit(&ctl->empty[st]);
        return true;
      };
      // O_X += P_X V_i, P_X from tensor memory (fp16 pairs over S_X).  (The
      // unit's first one overwrites O_X: the tile's warps have read the last
      // unit's before they wrote this P.)
      auto issue_pv = [&](int X, int i, bool begins, bool first, bool last) -> bool {
        if (!wait_bar(&ctl->p_full[X], pcnt[X] & 1)) return false;
        ++pcnt[X];
        const uint32_t m = 2 * (g + i) + 1;
        const int st = m % S;
        if (first && !wait_bar(&ctl->full[st], (m / S) & 1)) return false;
        tc_fence_after();
        const uint64_t b0 = desc_v + ((kv_addr + st * C::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_f16_ts(tmem + C::o_col(X), tmem + C::s_col(X) + kk * 8, b0 + ((kk * 16 * 128) >> 4), idesc_o,
                      (!begins || kk > 0) ? 1u : 0u);
        if (last) umma_commit(&ctl->empty[st]);
        return true;
      };
      if (share) {  // tile X of the rows takes key tiles X, X + 2, ...
        ok = issue_s(0, 0, true, true, true) && issue_s(1, 1, true, true, true);
        for (int i = 0; i < n && ok; ++i) {
          const int X = i & 1;
          ok = issue_pv(X, i, i < 2, true, true);
          if (!ok) break;
          if (i + 2 >= n) umma_commit(&ctl->o_done[X]);
          else ok = issue_s(X, i + 2, false, true, true);
        }
      } else {
        for (int X = 0; X <= last_x && ok; ++X) ok = issue_s(X, 0, true, X == 0, X == last_x);
        for (int i = 0; i < n && ok; ++i)
          for (int X = 0; X <= last_x && ok; ++X) {
            ok = issue_pv(X, i, i == 0, X == 0, X == last_x);
            if (!ok) break;
            if (i == n - 1) umma_commit(&ctl->o_done[X]);
            else ok = issue_s(X, i + 1, false, X == 0, X == last_x);
          }
      }
      g += n;
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
  } else if (warp >= kMakeWarp0) {
    // ------------------------------------------------------- operand K or V
    const bool is_v = warp >= kMakeWarp0 + 4;
    const int w4 = warp & 3, key_of_tile = w4 * 32 + lane;
    const uint8_t* pool = is_v ? p.value_cache : p.key_cache;
    const int run = q4_run_bytes(p.g.bs, D);
    // 16-byte unit of the row that storage chunk c, group j goes to: (4 (j %
    // 2) + c) ^ turn, the layout's and the tile's swizzles in one.
    const uint32_t turn = ((key_of_tile >> 2) & 3) ^ (key_of_tile & 7);
    const uint32_t row_addr = smem_u32(kv_s) + key_of_tile * 128;
    // Three tiles are in work: one's codes are in registers and being made,
    // the next one's are on their way, and the page of the one after is.
    uint32_t l_unit = 0;
    int l_i = 0, l_n = 0, f_h = 0, f_key = 0, f_page = -1;
    bool l_end = false, f_in = false;
    // Finds the tile after the last one found, this thread's key in it, and
    // asks for the key's page; false at the end.
    auto find = [&]() -> bool {
      while (!l_end && l_i == l_n) {
        const uint32_t s = l_unit % kInfoRing;
        if (!warp_wait(&ctl->info_full[s], (l_unit / kInfoRing) & 1, abort, p.g.err, p.err_site, kSite | 3) ||
            ctl->info[s].n == 0) {
          l_end = true;
        } else {
          l_i = ctl->info[s].i0;
          l_n = l_i + ctl->info[s].n;
          ++l_unit;
        }
      }
      if (l_end) return false;
      const Unit& u = ctl->info[(l_unit - 1) % kInfoRing];
      f_key = tile_key(u, l_i++) + key_of_tile;
      f_h = u.h;
      f_in = f_key <= u.pos_max && (f_key >= u.lo_min || f_key < p.first);
      if (f_in) f_page = p.g.block_table[(size_t)u.b * p.g.MB + (f_key >> p.g.log_bs)];
      return true;
    };
    // What the found tile's key is to this thread, and where its row is.
    enum { kNever, kUnmapped, kHeld };  // never admitted: zeros; no page: zeros and a mask
    int next_row = 0;
    size_t next_at = 0;
    auto resolve = [&]() -> int {
      if (!f_in) return kNever;
      if (f_page < 0 || f_page >= p.g.NB) {
        if (f_page != -1) atomicOr(p.g.err, PA_DEVERR_BLOCK_ID);
        return kUnmapped;
      }
      next_row = f_key & (p.g.bs - 1);
      next_at = ((size_t)f_page * p.g.Hk + f_h) * run;
      return kHeld;
    };
    uint4 codes[kGroups];
    unsigned short scales[kGroups];
    auto load = [&]() {
      const uint8_t* at = pool + next_at + next_row * (D / 2);
      const uint8_t* sc = pool + next_at + p.g.bs * (D / 2) + next_row * 2;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        codes[i] = *reinterpret_cast<const uint4*>(at + 16 * i);
        scales[i] = *reinterpret_cast<const unsigned short*>(sc + i * p.g.bs * 2);
      }
    };
    bool more = find();
    int state = more ? resolve() : kNever;
    if (state == kHeld) load();
    uint32_t unit = 0, tile = 0;
    bool found = more && find();
    while (more) {
      // Masks of the tile, before its scores are looked at.  A scale of V
      // that is no number leaves zeros; rows that admit the key know of it.
      bool held = state == kHeld;
      uint32_t bits = __ballot_sync(0xffffffffu, state == kUnmapped);
      if (is_v) {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) bad |= (scales[j] & 0x7c00) == 0x7c00;
        bad &= held;
        held &= !bad;
        bits = __ballot_sync(0xffffffffu, bad);
      }
      if (lane == 0) {
        TileMask& m = ctl->mask[tile % kMaskRing];
        (is_v ? m.bad : m.unmapped)[w4] = bits;
        mbar_arrive(&ctl->mask_full[tile % kMaskRing]);
      }
      const uint32_t n = 2 * tile + (is_v ? 1 : 0), slot = n % S;
      if (!warp_wait(&ctl->empty[slot], ((n / S) & 1) ^ 1, abort, p.g.err, p.err_site, kSite | 4)) break;
      const uint32_t to = row_addr + slot * C::kTileBytes;
#pragma unroll
      for (int wi = 0; wi < D / 8; ++wi) {
        const int c = wi / kGroups, j = wi % kGroups;
        const uint32_t words[4] = {codes[wi / 4].x, codes[wi / 4].y, codes[wi / 4].z, codes[wi / 4].w};
        uint4 y = make_uint4(0, 0, 0, 0);
        if (held) y = make_values(words[wi % 4], (uint32_t)scales[j] * 0x10001u);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (j >> 1) * (kTile * 128) +
                                                                      ((((j & 1) * 4 + c) ^ turn) << 4)),
                     "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                     : "memory");
      }
      // The next tile's codes on their way, and the page of the one after.
      more = found;
      const uint32_t unit_next = l_unit - 1;
      state = more ? resolve() : kNever;
      if (state == kHeld) load();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->full[slot]);
        if (!more || unit_next != unit) mbar_arrive(&ctl->info_empty[unit % kInfoRing]);
      }
      found = more && find();
      unit = unit_next;
      ++tile;
    }
  } else {
    regs_inc<kRegSoftmax>();
    // -------------------------------------- query operand, softmax, output
    const int X = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t scnt = 0, ocnt[2] = {0, 0}, bcnt = 0, g = 0;
    float2* b_sums = reinterpret_cast<float2*>(q_s + C::kTileBytes);  // (B's operand is free then)
    for (uint32_t tt = 0;; ++tt) {
      const int slot = tt % kInfoRing;
      if (!warp_wait(&ctl->info_full[slot], (tt / kInfoRing) & 1, abort, p.g.err, p.err_site, kSite | 5)) break;
      const Unit& ui = ctl->info[slot];
      const int n = ui.n;
      if (n == 0) break;
      const bool share = SHARE && shared_tile(ui);
      if (X == 1 && !share && ui.nrows <= kTile) {  // no tile B
        g += n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->info_empty[slot]);
        continue;
      }
      const int r_unit = share ? r : X * kTile + r;
      const bool row_ok = r_unit < ui.nrows;
      const int rho = ui.row0 + (row_ok ? r_unit : 0), tok = rho / p.G;
      const int head = ui.h * p.G + rho - tok * p.G, pos = ui.past + tok;
      const size_t row = (size_t)(ui.t0 + tok) * p.H + head;
      const int lo = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
      // The row as an operand (its tile is free: the last scores that it
      // gave have been read).
      float f = 0.f;
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.query + row * D);
        auto value = [&](uint32_t w, float* v) {
          if (p.bf16) {
            v[0] = __uint_as_float(w << 16);
            v[1] = __uint_as_float(w & 0xffff0000u);
          } else {
            const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&w));
            v[0] = h2.x;
            v[1] = h2.y;
          }
        };
        float top = 0.f;
#pragma unroll 1
        for (int i = 0; i < D / 8; i += 4) {
          uint4 raw[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) raw[k] = row_ok ? src[i + k] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v[2];
              value(w[e], v);
              top = max3(top, fabsf(v[0]), fabsf(v[1]));
            }
          }
        }
        const int up = top > 0.f && top < INFINITY ? 14 - ilogbf(top) : 0;
        const float up0 = __int_as_float((127 + up / 2) << 23), up1 = __int_as_float((127 + up - up / 2) << 23);
#pragma unroll 1
        for (int i = 0; i < D / 8; i += 2) {
          uint4 raw[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) raw[k] = row_ok ? src[i + k] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v[2];
              value(w[e], v);
              y[e] = pack_half2(v[0] * up0 * up1, v[1] * up0 * up1);
            }
            *reinterpret_cast<uint4*>(q_s + X * C::kTileBytes + ((i + k) >> 3) * (kTile * 128) + r * 128 +
                                      ((((i + k) & 7) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        // (8: the operands are eighths of the values)
        f = ldexpf(CAP ? 2.f * kLog2e * p.scale / p.softcap : p.scale * kLog2e, 3 - up);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[X]);

      float m_ref = -INFINITY, l = 0.f, back = 1.f;  // (back: what the row's scores were divided by)
      const int i_first = share ? X : 0, i_step = share ? 2 : 1;
      // B waits for the unit's first scores before its masks: a wait for masks
      // alone cannot tell a turn of their ring from the one two turns later,
      // and B, which skips units without a tile B, may be that far ahead of
      // the warps that write them.  With a tile's scores there, its K and every
      // V up to two tiles before it have been made, so this tile's masks and
      // the next ones' are at most a turn away.  A has had every unit's output
      // by then, which says as much.  (Scores before masks in each tile: the
      // chunks above take 631 us.)
      bool ok = X == 0 || warp_wait(&ctl->s_full[X], scnt & 1, abort, p.g.err, p.err_site, kSite | 7);
      if (!ok) break;
      for (int i = i_first; i < n; i += i_step) {
        const uint32_t tile = g + i;
        const int key0 = tile_key(ui, ui.i0 + i);
        if (!warp_wait(&ctl->mask_full[tile % kMaskRing], (tile / kMaskRing) & 1, abort, p.g.err, p.err_site, kSite | 6)) {
          ok = false;
          break;
        }
        const TileMask& tm = ctl->mask[tile % kMaskRing];
        const uint4 unmapped = *reinterpret_cast<const uint4*>(tm.unmapped), bad = *reinterpret_cast<const uint4*>(tm.bad);
        if (!warp_wait(&ctl->s_full[X], scnt & 1, abort, p.g.err, p.err_site, kSite | 7)) {
          ok = false;
          break;
        }
        ++scnt;
        tc_fence_after();
        const int c_hi = row_ok ? pos - key0 : kTile - 1, c_lo = row_ok ? lo - key0 : 0, c_f = p.first - key0;
        bool spoilt = false;  // admits a key whose V is no number
        float alpha = 1.f;    // what the references' moves make of the sums so far
        float sum = 0.f;      // of this tile's weights
        // In two halves, for the registers' sake: the second may move the
        // reference too, and takes the first's weights along then.  A loop
        // where the tile is shared (unrolled, 36 rows take 144 us, not 135),
        // unrolled elsewhere (as a loop, the chunks take 630 us).
#pragma unroll(SHARE ? 1 : 2)
        for (int half = 0; half < 2; ++half) {
          const uint32_t gone[2] = {half ? unmapped.z : unmapped.x, half ? unmapped.w : unmapped.y};
          const uint32_t no_v[2] = {half ? bad.z : bad.x, half ? bad.w : bad.y};
          constexpr int kKeys = kTile / 2;
          float x[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) tmem_ld32(lane_addr + C::s_col(X) + half * kKeys + c, x + c);
          tmem_ld_wait();
          if constexpr (CAP) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) x[c] = p.softcap * kLog2e * (1.f - 2.f * rcp(1.f + ex2(x[c] * f)));
          }
          const int h_hi = c_hi - half * kKeys, h_lo = c_lo - half * kKeys, h_f = c_f - half * kKeys;
          if (h_hi < kKeys - 1 || (h_lo > 0 && h_f < kKeys)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) x[c] = c <= h_hi && (c >= h_lo || c < h_f) ? x[c] : -INFINITY;
          }
          if (gone[0] | gone[1]) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) x[c] = (gone[c >> 5] >> (c & 31)) & 1 ? -INFINITY : x[c];
          }
          if (no_v[0] | no_v[1]) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) spoilt |= ((no_v[c >> 5] >> (c & 31)) & 1) && x[c] != -INFINITY;
          }
          const float cand = max_tree<kKeys>(x) * (CAP ? 1.f : f);
          float up = 1.f;
          if (cand > __fadd_rd(m_ref, kLift + kSlack) || (m_ref == -INFINITY && cand != -INFINITY)) {
            float to = ceilf(cand) - kLift;
            up = __int_as_float((127 + max(__float2int_rn(m_ref - to), -127)) << 23);  // 2^(m_ref - to), 0 below 2^-126
            // Past 2^24 a rounded reference lies further from the unrounded
            // products below than the weights' exponents reach: the row's
            // scores are taken in larger units from here on, in which the
            // largest is below 2^24 and keys that differ at all in fp32
            // still hardly share a weight.
            const int by = (int)(__float_as_uint(cand) << 1 >> 24) - (127 + 23);  // (above 104: no number)
            if (!CAP && by > 0 && by <= 104) {
              const float down = __int_as_float((127 - by) << 23);
              f *= down;
              back *= __int_as_float((127 + by) << 23);
              to = ceilf(cand * down) - kLift;
            }
            m_ref = to;
            alpha *= up;
          }
          const float mul = CAP ? 1.f : f;
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          __syncwarp();
          if (half == 1 && __any_sync(0xffffffffu, up != 1.f)) {
            uint32_t pk[32];
            tmem_st_wait();
            tmem_ld32(lane_addr + C::s_col(X), reinterpret_cast<float*>(pk));
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&pk[q]));
              pk[q] = pack_half2(w.x * up, w.y * up);
            }
            tmem_st16(lane_addr + C::s_col(X), pk);
            tmem_st16(lane_addr + C::s_col(X) + 16, pk + 16);
          }
          const uint64_t mul2v = f2(mul, mul), neg_m2 = f2(-m_use, -m_use);
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < kKeys; h += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const uint64_t arg = fma2(f2(x[h + 2 * q], x[h + 2 * q + 1]), mul2v, neg_m2);
              float a0, a1;
              unf2(arg, a0, a1);
              const float e0 = ex2(a0), e1 = ex2(a1);
              sum2[q & 1] = add2(sum2[q & 1], f2(e0, e1));
              pk[q] = pack_half2(e0, e1);
            }
            // P_X -> TMEM over S_X: 32 keys as 16 columns of fp16 pairs
            tmem_st16(lane_addr + C::s_col(X) + half * (kKeys / 2) + h / 2, pk);
          }
          float a0, a1;
          unf2(add2(sum2[0], sum2[1]), a0, a1);
          sum = sum * up + (a0 + a1);
        }
        if (i > i_first && __any_sync(0xffffffffu, alpha != 1.f)) {
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[X]);
        l = l * alpha + sum;
        if (spoilt) l = __int_as_float(0x7fffffff);
      }
      g += n;
      if (!ok) break;
      if constexpr (!CAP) m_ref *= back;
      if (share && X == 1) {  // A joins
        ++ocnt[1];
        b_sums[r] = make_float2(m_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->b_ready);
        if (!warp_wait(&ctl->b_taken, bcnt & 1, abort, p.g.err, p.err_site, kSite | 9)) break;
        ++bcnt;
        if (lane == 0) mbar_arrive(&ctl->info_empty[slot]);
        continue;
      }
      if (!warp_wait(&ctl->o_done[X], ocnt[X] & 1, abort, p.g.err, p.err_site, kSite | 8)) break;
      ++ocnt[X];
      float mine = 1.f, other = 0.f;  // what A's and B's output are multiplied by
      if (X == 0 && ui.nrows > kTile) ++ocnt[1];
      if (share) {
        if (!warp_wait(&ctl->b_ready, bcnt & 1, abort, p.g.err, p.err_site, kSite | 10)) break;
        if (!warp_wait(&ctl->o_done[1], ocnt[1] & 1, abort, p.g.err, p.err_site, kSite | 11)) break;
        ++bcnt;
        ++ocnt[1];
        const float2 b = b_sums[r];
        const float top = fmaxf(m_ref, b.x);
        if (top != -INFINITY) {
          mine = m_ref == -INFINITY ? 0.f : ex2(m_ref - top);
          other = b.x == -INFINITY ? 0.f : ex2(b.x - top);
          m_ref = top;
        }
        l = l * mine + b.y * other;
      }
      tc_fence_after();
      // Output: O times 8 over the sum, or the partial results.
      float inv = 0.f;
      const size_t at = ui.part < 0 ? 0 : (size_t)ui.part * kQ4TileRows + r_unit;
      if (ui.part < 0) {
        float den = l;
        if (p.head_sink && m_ref != -INFINITY)
          den += ex2(elem16_to_float(p.head_sink[head], p.bf16) * kLog2e - m_ref);
        inv = m_ref == -INFINITY && l == 0.f ? 0.f : 8.f / den;
      } else if (row_ok) {
        p.tile_ml[at] = make_float2(l == 0.f ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref, l);
      }
      __half* dst = p.out + row * D;
      float4* part = reinterpret_cast<float4*>(p.tile_o) + (size_t)(ui.part < 0 ? 0 : ui.part) * (D / 4) * kQ4TileRows + r_unit;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tmem_ld32(lane_addr + C::o_col(X) + 32 * c, o);
        if (share) {
          float o1[32];
          tmem_ld32(lane_addr + C::o_col(1) + 32 * c, o1);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = o[e] * mine + o1[e] * other;
        }
        tmem_ld_wait();
        if (row_ok && ui.part < 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = o[8 * q + 2 * e] * inv, b = o[8 * q + 2 * e + 1] * inv;
              w[e] = p.bf16 ? pack_bf162(a, b) : pack_half2(a, b);
            }
            *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (row_ok) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            part[(size_t)(8 * c + q) * kQ4TileRows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
        __syncwarp();
      }
      // (the next P, after this, lets the tensor core overwrite O)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (share) mbar_arrive(&ctl->b_taken);
        mbar_arrive(&ctl->info_empty[slot]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch_d(const Q4Params& p, bool configure, cudaStream_t s) {
  static_assert(Cfg<D>::kSlots >= 4 && Cfg<D>::kSlots / 2 + 2 <= kMaskRing, "ring");
  const bool cap = p.softcap > 0.f;
  auto plain = cap ? q4_tile_kernel<D, true, false> : q4_tile_kernel<D, false, false>;
  auto share = cap ? q4_tile_kernel<D, true, true> : q4_tile_kernel<D, false, true>;
  if (configure) {
    const cudaError_t e = cudaFuncSetAttribute(plain, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(share, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  }
  // Which of the two is a rule on the mean, since only the device knows each
  // sequence's rows; both take any.
  const bool few = (long long)p.g.T * p.G <= (long long)kTile * p.g.batch;
  return launch_pdl(few ? share : plain, dim3(p.num_sms), kThreads, Cfg<D>::kSmem, s, p);
}

}  // namespace

cudaError_t q4_tile_configure(int D, float softcap) {
  Q4Params p{};
  p.softcap = softcap;
  return D == 64 ? launch_d<64>(p, true, nullptr) : launch_d<128>(p, true, nullptr);
}

cudaError_t launch_q4_tile(const Q4Params& p, cudaStream_t s) {
  return p.g.D == 64 ? launch_d<64>(p, false, s) : launch_d<128>(p, false, s);
}

}  // namespace pa
