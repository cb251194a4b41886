// Internal structures of the tree operators (rotary at explicit positions,
// attention for trees of drafted tokens, commit of the accepted path).
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pa.h"

namespace pa {

// ---- shared host helpers (api.cu)
// Records the thread's last message (pa_last_error_message(NULL)) and returns st.
pa_status host_fail(pa_status st, const char* fmt, ...);
// 3-D view {D, heads_total, rows_total} of rows of heads, box {64, heads_box, rows_box}, 128-byte swizzle.
bool encode_rows_map(CUtensorMap* m, const void* base, int D, int heads_total, long long rows_total, int heads_box,
                     int rows_box);
// 5-D view {64 channels, 8 rows, D/64 chunks, rows_total/8 groups, Hk} of a pool: a box {64, 8, D/64, rows_box/8, 1}
// is one head's rows laid out [group][chunk][row][128 B] with the 128-byte swizzle.
bool encode_groups_map(CUtensorMap* m, const void* base, int D, int Hk, long long rows_total, int rows_box);

// ---- rotary (rotary.cu)
constexpr int kRotaryMaxHeads = 4096;
struct RotaryRows {  // rows of one tensor; nheads == 0: absent
  const void* src;
  void* dst;           // NULL for rows that go to the pool
  long long src_stride, dst_stride;  // elements
  int nheads;
};

struct RotaryParams {
  RotaryRows q, k, v;  // v: copied rows (pool mode only)
  const unsigned long long* steps;
  const int* positions;
  int T;
  int D, R, off;
  float factor, sin_sign;
  int parts;           // warps per token, each a contiguous share of the token's head items
  // pool mode (key_cache != NULL): K and V rows to slots of the paged pool
  void* key_cache;
  void* value_cache;
  const int* block_table;
  const int* cum;
  const int* past;
  int batch, bs, NB, MB;
  int* err;
};
cudaError_t launch_rotary(const RotaryParams& p, int dtype, int interleaved, cudaStream_t s);

// ---- commit (tree_commit.cu)
constexpr int kCommitLayers = 128;  // layers of one launch
struct CommitParams {
  void* pools[2 * kCommitLayers];   // K, V, K, V, ...
  int n_pools;
  int row_vecs;                     // 16-byte vectors of one slot's row
  const int* block_table;
  const int* past;
  const int* accepted;
  const int* count;
  int max_accepted, max_draft, batch, bs, NB, MB;
  int* new_past;
  int* err;
};
cudaError_t launch_commit(const CommitParams& p, int num_sms, cudaStream_t s);

// ---- tree attention (tree_attention.cu)
constexpr int kTreeMaxDraft = 256;
constexpr int kTreeMaxWords = kTreeMaxDraft / 32;

// A unit of work whose partial results lie in several chunks' slots.
struct Cut {
  int rows;          // rows of the unit's partial results
  int slot0, slot1;  // slots of the first and second partial; later ones are 2 Hk slots further each
  int more;          // partials behind the first
  int t0, ntok, k;
  int pad;
};

struct TreeCounters {  // zero between calls
  int n_cuts[2];  // units in two pieces, in more
  int joined;   // blocks of the joining kernel that are done
};

struct TreeParams {
  const __half* value_cache;
  const int* block_table;
  const int* cum;
  const int* past;
  const int* positions;      // NULL: past + j
  const uint32_t* mask;      // NULL: causal
  const float* slopes;       // NULL: none
  const __half* head_sink;   // NULL: none
  __half* out;
  int batch, T;
  int H, Hk, G, D;
  int tile_tokens;           // tokens of a row tile (128 / rep rows)
  int unit_tokens;           // tokens of a unit: two row tiles, or one (head_size 256)
  int inv_unit;              // 2^20 / unit_tokens, rounded up
  int bs, NB, MB, log_bs, log_page_rows, oob_row;
  int max_draft, words, max_kv;
  int window;
  int n_ranges;              // ranges of the line at most
  int q_tiles;               // 2 when a unit may have two row tiles
  int rep;                   // replicas of the rows (1, 2 or 4)
  float scale, softcap;
  // workspace
  TreeCounters* counters;
  Cut* cuts;                 // [chunks]
  float2* part_ml;           // [2 chunks][part_rows]
  float4* part_o;            // [2 chunks][D / 4][part_rows]
  int* groups;               // [CTAs][n_groups]: starts of the groups of 32 sequences (batches beyond one block)
  int n_groups;              // groups of this call
  int part_rows;
  int* err;
  int* err_site;
};
template <int D>
cudaError_t tree_configure(int bf16, int rep);
template <int D>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                        int bf16, int grid, cudaStream_t s);
template <> cudaError_t tree_configure<64>(int, int);
template <> cudaError_t tree_configure<128>(int, int);
template <> cudaError_t tree_configure<256>(int, int);
template <> cudaError_t launch_tree<64>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const TreeParams&,
                                        int, int, cudaStream_t);
template <> cudaError_t launch_tree<128>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const TreeParams&,
                                         int, int, cudaStream_t);
template <> cudaError_t launch_tree<256>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const TreeParams&,
                                         int, int, cudaStream_t);

}  // namespace pa
