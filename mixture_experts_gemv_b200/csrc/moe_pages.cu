// moe_pages.cu -- copies of cache pages: page dst[i] = page src[i] of K and V in every layer, and,
// for a move, the block-table entries that name a source page.
//
// Bound: HBM (every byte of the pages read and written once). The list of pairs travels in the
// kernel's parameters, so a call needs no device buffer and no copy of its own, and a captured
// launch holds its list. A block copies a 16 KB stretch of one page of one layer's K or V, four
// 16-byte pieces a thread, all loads in flight before the stores. Sources and destinations are
// disjoint (checked on the host), so the order of blocks does not matter. The table's blocks come
// first in the grid and run beside the copies: each entry is looked up in the sorted sources.
//
// Measured (8 KV heads of 256, bf16, pages of 16): 601 pages of 5 layers and 32 rows of tables,
// 788 MB moved, 120.0 us = 6.57 TB/s (a plain copy's rate); 8 pages of 30 layers, 63 MB, 11.1 us
// = 5.7 TB/s, 1.5 us above the bytes: the launch and the first blocks' loads.
#include "moe_attn.cuh"
#include "moe_pages.cuh"

namespace {

constexpr int kThreads = 256, kPer = 4;
constexpr int kFewPairs = 256, kManyPairs = 3968;   // lists of 2 KB and 31 KB: the parameter limit is 32,764 bytes

template <int N> struct Pairs {
  int2 v[N];   // (src, dst), ascending src
};

template <int N, bool DENSE>
__global__ void __launch_bounds__(kThreads) k_copy_pages(const __grid_constant__ CopyParams p, const __grid_constant__ Pairs<N> list) {
  const int tid = threadIdx.x;
  long long block = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (block < p.table_blocks) {
    __shared__ int src[N];
    for (int i = tid; i < p.n; i += kThreads) src[i] = list.v[i].x;
    __syncthreads();
    const long long entries = (long long)p.rows * p.cols;
    for (long long e = block * kThreads + tid; e < entries; e += (long long)p.table_blocks * kThreads) {
      const long long r = e / p.cols;
      int32_t *at = p.tables + r * p.table_stride + (e - r * p.cols);
      const int page = *at;
      int lo = 0, hi = p.n;   // first source that is not below the entry
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (src[mid] < page) lo = mid + 1;
        else hi = mid;
      }
      if (lo < p.n && src[lo] == page) *at = list.v[lo].y;
    }
    return;
  }
  block -= p.table_blocks;
  // (layer, K or V, pair, stretch of the page)
  const long long rest = block / p.stretches;
  const int stretch = (int)(block - rest * p.stretches);
  const int pair = (int)(rest % p.n);
  const int lk = (int)(rest / p.n), layer = lk >> 1;
  char *base = (lk & 1 ? p.v : p.k) + layer * p.layer_b;
  const int2 sd = list.v[pair];
  const char *from = base + sd.x * p.page_b;
  char *to = base + sd.y * p.page_b;
  uint4 w[kPer];
  long long at[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    long long i = (long long)stretch * (kThreads * kPer) + j * kThreads + tid;   // 16-byte piece of the page
    at[j] = -1;
    if (i < p.pieces) {
      if (DENSE) {
        at[j] = i * 16;
      } else {
        const long long run = i / p.run_pieces, a = run / p.inner;
        at[j] = a * p.outer_b + (run - a * p.inner) * p.inner_b + (i - run * p.run_pieces) * 16;
      }
      w[j] = __ldcs(reinterpret_cast<const uint4 *>(from + at[j]));
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (at[j] >= 0) __stcs(reinterpret_cast<uint4 *>(to + at[j]), w[j]);
}

template <int N, bool DENSE> int launch_part(CopyParams p, const int2 *pairs, cudaStream_t s) {
  Pairs<N> list;
  for (int i = 0; i < p.n; ++i) list.v[i] = pairs[i];
  const long long blocks = p.table_blocks + (long long)p.stretches * p.n * p.layers * 2;
  PdlLaunch l(dim3((unsigned)blocks), kThreads, 0, s);
  if (cudaLaunchKernelEx(&l.cfg, k_copy_pages<N, DENSE>, p, list) != cudaSuccess) return -1;
  moe_prof_count(1);
  return 0;
}

}  // namespace

int moe_launch_copy_pages(CopyParams p, const int2 *pairs, int n, cudaStream_t s) {
  const bool dense = p.run_pieces == p.pieces;
  p.table_blocks = 0;
  if (p.tables) {
    const long long want = ((long long)p.rows * p.cols + kThreads - 1) / kThreads;
    p.table_blocks = (int)(want < 592 ? want : 592);   // up to four blocks an SM
  }
  const long long stretches = (p.pieces + kThreads * kPer - 1) / (kThreads * kPer);
  if (p.table_blocks + (double)stretches * (n < kManyPairs ? n : kManyPairs) * p.layers * 2 > 2147483647.0) return -2;
  p.stretches = (int)stretches;
  // lists above the parameter limit run as several launches: the pairs are independent of each
  // other, and no destination is another pair's source, so a table entry moves once
  for (int i = 0; i < n; i += kManyPairs) {
    p.n = n - i < kManyPairs ? n - i : kManyPairs;
    const int rc = p.n <= kFewPairs
                       ? (dense ? launch_part<kFewPairs, true>(p, pairs + i, s) : launch_part<kFewPairs, false>(p, pairs + i, s))
                       : (dense ? launch_part<kManyPairs, true>(p, pairs + i, s) : launch_part<kManyPairs, false>(p, pairs + i, s));
    if (rc) return rc;
  }
  return 0;
}
