"""q, k, v and outputs whose heads lie between each other's in one buffer."""
import pytest
import torch

import mixture_experts_gemv_b200 as moe
from test_gpu_attention import BF, DEV, FP, _built, gen, make_batch, make_cache, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_heads_of_q_k_and_v_in_turn_turned_in_place(T, dtype):
    g = gen(T)
    H, D = 8, 96
    qkv = normal((T, H, 3, D), dtype, g)
    q, k, v = qkv.unbind(2)
    pos = torch.arange(T, device=DEV, dtype=torch.int32) + 50
    inv, _ = moe.moe_rope_frequencies(64, device=DEV)
    gain = torch.randn(D, generator=g, device=DEV)
    slots = torch.randperm(T + 40, generator=g, device=DEV)[:T]
    pages = -(-(T + 40) // 16)
    args = dict(q_gain=gain, k_gain=gain, slots=slots)
    apart, here = make_cache(pages, 16, H, D, dtype, "HND", g), make_cache(pages, 16, H, D, dtype, "HND", g)
    q_out, k_out, v_was = torch.empty_like(q), torch.empty_like(k), v.clone()
    moe.moe_qk_norm_rope(q.contiguous(), k.contiguous(), v.contiguous(), pos, inv, q_out=q_out, k_out=k_out, cache=apart, **args)
    moe.moe_qk_norm_rope(q, k, v, pos, inv, q_out=q, k_out=k, cache=here, **args)
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(v, v_was)
    for a, b in ((apart.k, here.k), (apart.v, here.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    moe.moe_cache_check()


def test_attention_output_between_the_heads_of_q():
    cache, tables, n, g = make_batch([300, 0, 41], 16, 2, 64, BF, "NHD", seed=3)
    both = normal((3, 8, 2, 64), BF, g, 2.0)
    q, out = both.unbind(2)
    want, was = torch.empty((3, 8, 64), device=DEV, dtype=BF), q.clone()
    moe.moe_attention_decode(q.contiguous(), cache, tables, n, want, 0.125)
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125)
    assert torch.equal(out, want) and torch.equal(q, was)
    moe.moe_cache_check()
