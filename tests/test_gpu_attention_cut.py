"""One-token attention whose sequences are cut over whole blocks, for every shape that the kernel is compiled for: the
blocks then join their warps' pieces before the join kernel does. Against the 64-bit form."""
import pytest
import torch

import mixture_experts_gemv_b200 as moe
from test_gpu_attention import BF, DEV, E4, FP, _built, check_attention, make_batch, normal  # noqa: F401

pytestmark = pytest.mark.gpu

# n_q, n_kv, D: every width (64, 128, 256, 512) with every number of column tiles of 8 heads, groups and widths that do
# not fill them, and a group that takes two passes over its KV head
SHAPES = [
    (16, 2, 64), (32, 2, 64), (40, 2, 48), (64, 2, 64), (71, 1, 64), (128, 2, 16),
    (8, 2, 128), (26, 2, 112), (64, 2, 128), (40, 1, 80),
    (14, 2, 256), (32, 2, 240), (8, 2, 512), (22, 2, 400),
]


WORKERS = 1792   # the most warps that a call's work is cut over


@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("nq,nkv,D", SHAPES)
def test_blocks_join_their_pieces(nq, nkv, D, dtype, cache_dtype):
    # two units of at most 32 tokens a warp: a block's warps then work on neighbouring ones. The longest sequence is
    # cut over many blocks
    lens = [75001, 0, 43000, 17] if nkv == 1 else [37003, 0, 21000, 17]
    units = sum(n // 32 for n in lens) * nkv
    assert units >= 2 * WORKERS and lens[0] // 32 >= 40 * (units // WORKERS)
    cache, tables, n, g = make_batch(lens, 16, nkv, D, cache_dtype, "NHD", seed=nq + D)
    q = normal((len(lens), nq, D), dtype, g, 2.0)
    out, lse = torch.full_like(q, float("nan")), torch.full((len(lens), nq), float("nan"), device=DEV)
    scale = D ** -0.5
    moe.moe_attention_decode(q, cache, tables, n, out, scale, lse=lse)
    check_attention(q, cache, tables, n, scale, 0, out, lse)
    again, lse2 = torch.full_like(q, float("nan")), torch.full_like(lse, float("nan"))
    moe.moe_attention_decode(q, cache, tables, n, again, scale, lse=lse2)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    moe.moe_cache_check()
