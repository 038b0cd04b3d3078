"""The join of a cut sequence's pieces behind a kernel that changes the lengths: the join starts while that kernel runs, and
has to follow what stands there when it has ended, whatever it read before."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include <vector>
#include "moe_attn_core.cuh"

// Lets the next kernel start, and writes the length some time later.
__global__ void k_write_late(int *lens, int length, long long clocks) {
  pdl_launch_dependents();
  const long long from = clock64();
  for (int i = 0; i < (1 << 20) && clock64() - from < clocks; ++i) __nanosleep(200);
  *lens = length;
}

// One sequence of one KV head of 64, 8 query heads, `before` tokens and then `length`, in units of 32 over 592 workers;
// every byte of the workspace that is not its pieces is NaN. Returns the largest error against the pieces' mean, or, where
// there is nothing to join, against untouched rows.
static float run(int before, int length, int par) {
  const int units = (length + 31) / 32, extra = units + 1 >= 2 * 592, w0 = 0, w1 = units < 592 ? (units > 0 ? units - 1 : 0) : 591;
  const int D = 64, nt = 1, workers = 592, frags = D / 16 * nt * 32, threads = par > 4 ? 512 : 256;
  float4 *o, *ml;
  int4 *cut;
  int *lens, *tables;
  __nv_bfloat16 *out;
  float *lse;
  uint32_t *err;
  cudaMalloc(&o, 2ll * workers * frags * 16);
  cudaMalloc(&ml, 2ll * workers * 4 * nt * 16);
  cudaMalloc(&cut, workers * sizeof(int4));
  cudaMalloc(&lens, 4);
  cudaMalloc(&tables, 4);
  cudaMalloc(&out, 8 * D * 2);
  cudaMalloc(&lse, 32);
  cudaMalloc(&err, 4);
  cudaMemset(o, 255, 2ll * workers * frags * 16);
  cudaMemset(ml, 255, 2ll * workers * 4 * nt * 16);
  cudaMemset(out, 0, 8 * D * 2);
  cudaMemset(err, 0, 4);
  cudaMemcpy(lens, &before, 4, cudaMemcpyHostToDevice);
  cudaMemset(cut, 255, workers * sizeof(int4));
  int pieces = 0;
  float sum = 0;
  for (int w = w0; w <= w1 && w1 > w0; ++w) {
    // a block of four workers strictly inside leaves one piece, its first worker's, where blocks join
    const int first = w / 4 * 4;
    if (extra && first > w0 && first + 3 < w1 && w != first) continue;
    const float value = 1 + pieces % 7;
    std::vector<float4> a(frags, make_float4(value, value, value, value)), m(4 * nt, make_float4(0, 1, 0, 1));
    const long long at = 2ll * w + (w == w0);
    cudaMemcpy(o + at * frags, a.data(), frags * 16, cudaMemcpyHostToDevice);
    cudaMemcpy(ml + at * 4 * nt, m.data(), 4 * nt * 16, cudaMemcpyHostToDevice);
    sum += value;
    ++pieces;
  }
  AttnParams p{};
  p.tables = tables;
  p.table_stride = 1;
  p.max_tokens = 1 << 30;
  p.lens = lens;
  p.B = 1, p.nq = 8, p.nkv = 1, p.D = D, p.group = 8, p.n_groups = 1;
  p.page_size = 1 << 30, p.page_shift = 30, p.num_pages = 1;
  p.v_scale = 1;
  p.out = out, p.out_tok = 8 * D, p.out_head = D;
  p.lse = lse;
  p.ws_o = reinterpret_cast<float *>(o);
  p.ws_ml = reinterpret_cast<float2 *>(ml);
  p.ws_cut = cut;
  p.by_segment = 1;
  p.err = err;
  const int per = threads / par;
  const size_t smem = par > 1 ? threads * 32 : 0;
  const dim3 grid(1, (frags + per - 1) / per);
  cudaStream_t stream;
  cudaStreamCreate(&stream);
  cudaDeviceSynchronize();
  {
    PdlLaunch l(dim3(1), 1, 0, stream);
    cudaLaunchKernelEx(&l.cfg, k_write_late, lens, length, 200000ll);   // about 100 us
  }
  {
    PdlLaunch l(grid, threads, smem, stream);
    cudaLaunchKernelEx(&l.cfg, moe_attn::k_attn_join<__nv_bfloat16, 2, false>, p, 5, workers, nt, par);
  }
  cudaStreamSynchronize(stream);
  cudaStreamDestroy(stream);
  std::vector<__nv_bfloat16> got(8 * D);
  if (cudaMemcpy(got.data(), out, 8 * D * 2, cudaMemcpyDeviceToHost) != cudaSuccess) return INFINITY;
  const float want = pieces ? sum / pieces : 0;
  float worst = 0;
  for (auto x : got) {
    const float off = fabsf(__bfloat162float(x) - want);
    if (!(off <= worst)) worst = off;
  }
  for (void *x : {(void *)o, (void *)ml, (void *)cut, (void *)lens, (void *)tables, (void *)out, (void *)lse, (void *)err}) cudaFree(x);
  return worst / (want > 0 ? want : 1);
}

int main() {
  const int lengths[] = {0, 32, 64, 320, 5000, 32 * 592, 32 * 592 * 3, -7};
  for (int par : {2, 4, 8, 16})
    for (int before : lengths)
      for (int length : lengths) printf("%d %d %d %g\n", par, before, length, run(before, length, par));
  return 0;
}
"""


def test_the_join_follows_the_lengths_behind_its_wait(tmp_path):
    (tmp_path / "join.cu").write_text(PROGRAM)
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "mixture_experts_gemv_b200", "csrc"),
                    "-o", str(tmp_path / "join"), str(tmp_path / "join.cu")], check=True)
    out = subprocess.run([str(tmp_path / "join")], check=True, capture_output=True, text=True, timeout=120).stdout
    rows = [line.split() for line in out.splitlines()]
    assert len(rows) == 4 * 8 * 8
    # the mean of the pieces, rounded to bf16 (half a step) after 32-bit sums
    bad = [r for r in rows if not float(r[-1]) <= 2.0 ** -8 * 1.01]
    assert not bad, bad[:20]
