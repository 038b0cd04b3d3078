// moe_pages.cuh -- parameters of the page-copy kernel.
#pragma once

#include "moe_common.cuh"

// A page is outer x inner runs of contiguous bytes (1 x 1 where the page is dense).
struct CopyParams {
  char *k, *v;
  int layers, n;
  long long layer_b, page_b, outer_b, inner_b;   // bytes
  int inner;                                     // runs per outer step
  long long run_pieces, pieces;                  // 16-byte pieces of a run, of a page
  int stretches;                                 // blocks a page (set by the launcher)
  int32_t *tables;
  long long table_stride;
  int rows, cols, table_blocks;
};

// pairs: n (src, dst), ascending src where p.tables is set. 0, -1 after a CUDA error, -2 when
// the grid would be too large.
int moe_launch_copy_pages(CopyParams p, const int2 *pairs, int n, cudaStream_t s);
