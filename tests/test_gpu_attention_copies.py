"""Two copies of the library in one process, as when a newer one is loaded beside it."""
import os
import shutil
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path.insert(0, %r)
import torch
import mixture_experts_gemv_b200 as moe
from mixture_experts_gemv_b200 import _lib

k = torch.randn(8, 16, 2, 128, device="cuda", dtype=torch.bfloat16); v = torch.randn_like(k)
cache = moe.MoeKvCache(k, v)
t = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
n = torch.tensor([60, 9], device="cuda", dtype=torch.int32)
q = torch.randn(2, 4, 128, device="cuda", dtype=torch.bfloat16)
outs = []
for path in (_lib.LIB_PATH, %r):
    _lib._lib, _lib.LIB_PATH = None, path
    out = torch.zeros_like(q)
    moe.moe_attention_decode(q, cache, t, n, out, 0.1)
    moe.moe_cache_check()
    outs.append(out)
assert torch.equal(*outs) and outs[0].abs().sum() > 0
print("fine")
"""


def test_two_copies_of_the_library(tmp_path):
    from mixture_experts_gemv_b200 import _lib, build
    build.build()
    other = str(tmp_path / "libmoe_other.so")
    shutil.copy(_lib.LIB_PATH, other)
    r = subprocess.run([sys.executable, "-c", CODE % (ROOT, other)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
