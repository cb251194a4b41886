// Internal structures of the operators over the pages of a cache.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pa.h"

namespace pa {

constexpr int kPagePools = 240;  // pools of one launch (a parameter's size)

// Results of a plan, in the handle's workspace.
struct PagePlan {
  int* n_moves;
  int2* moves;     // (source page, destination page), [num_blocks]; a negative source is left out
  int* free_list;  // [num_blocks]
  int* place;      // [num_blocks]: a page's new place (compact), marks (copy), counts before the call (resize)
  int* first;      // [max_rows]: first child of a row (fork)
  int* entries;    // [max_rows]: entries of a new row (fork); -1: the row failed (resize)
  int* fresh;      // [max_rows]: a row's own last page or -1 (fork); where its pages start in free_list (resize)
};

struct PagesParams {
  PagePlan w;
  int bs, NB, MB, rows_in, rows;
  const int* table;      // [rows_in, MB]
  int* table_out;        // [rows, MB]
  const int* lengths;    // [rows_in]
  int* lengths_out;      // [rows]
  const int* parent;     // fork
  const int* delta;      // resize
  const int* ref;        // [NB]
  int* ref_out;
  int* live;             // compact
  const int* src;        // copy
  const int* dst;
  int n_pairs;
  int* err;
};

struct PageCopyParams {
  void* pools[kPagePools];
  int n_pools;
  int with_tables;       // this launch also writes the tables and counts
  long long page_vecs;   // 16-byte vectors of a page
};

enum PageOp { kPageCopy = 0, kPageFork = 1, kPageResize = 2, kPageCompact = 3 };
cudaError_t launch_page_plan(PageOp op, const PagesParams& p, cudaStream_t s);
cudaError_t launch_page_apply(PageOp op, const PagesParams& p, const PageCopyParams& c, int num_sms, cudaStream_t s);

}  // namespace pa
