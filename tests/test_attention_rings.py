"""The shared memory of the one-token attention kernel, without a GPU: its compile-time shapes, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(64, 1), (64, 2), (64, 4), (64, 8), (128, 1), (128, 2), (128, 4), (256, 1), (256, 2), (512, 1)]   # width, column tiles

PROGRAM = """
#include <cstdio>
#include "moe_attn_core.cuh"
template <int W, int NT, int ES> void row() {
  using S = moe_attn::Shape<W, NT, ES>;
  printf("%%d %%d %%d %%d %%d %%d\\n", W, NT, ES, S::kUnit, S::kSlots, S::kSmem);
}
int main() {
%s
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """{(width, tiles, bytes an element): (bytes of a unit, slots, shared memory of a block)}"""
    at = tmp_path_factory.mktemp("rings")
    rows = "\n".join(f"  row<{w}, {nt}, {es}>();" for w, nt in SHAPES for es in (1, 2))
    (at / "shapes.cu").write_text(PROGRAM % rows)
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "mixture_experts_gemv_b200", "csrc"),
                    "-o", str(at / "shapes"), str(at / "shapes.cu")], check=True)
    out = subprocess.run([str(at / "shapes")], check=True, capture_output=True, text=True).stdout
    got = {}
    for line in out.splitlines():
        w, nt, es, *rest = map(int, line.split())
        got[w, nt, es] = rest
    return got


@pytest.mark.parametrize("es", [1, 2])
@pytest.mark.parametrize("w,nt", SHAPES)
def test_a_warps_ring_holds_its_copies_and_its_staged_rows(shapes, w, nt, es):
    unit, slots, smem = shapes[w, nt, es]
    ring = unit * slots
    assert unit % (16 * w * es) == 0              # whole tiles of 16 rows
    assert slots >= 3                             # K and V of the unit at hand, and one copy ahead
    assert ring >= w * nt * 8 * 4                 # 8 heads a column tile, FP32: what a joining block stages
    assert smem == 4 * ring and smem + 4 * 4 * nt * 16 <= 232448 - 1024   # four warps, and their maxima and sums
