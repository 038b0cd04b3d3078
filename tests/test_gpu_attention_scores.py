"""One-token attention at scores far beyond what the steps of 32-bit numbers resolve, against the 64-bit form."""
import pytest
import torch

import attn_ref as ref
import mixture_experts_gemv_b200 as moe
from test_gpu_attention import BF, DEV, E4, FP, _built, check_attention, make_batch, normal  # noqa: F401

pytestmark = pytest.mark.gpu
LN2 = 0.693147182464599609375   # ln 2 in 32 bits: times log2 e it rounds to 1, so scores in base 2 stay whole numbers


@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("power", [10, 23, 24, 25, 26, 27, 28, 29, 40, 60])
@pytest.mark.parametrize("lens,nkv,D", [([1, 40, 700, 5000], 1, 64), ([60000, 0, 33], 2, 128)])   # few units; blocks that join
def test_scores_of_any_size(lens, nkv, D, power, dtype, cache_dtype):
    """Scores (in base 2) of +-2^power plus a few of its steps: q . k = +-2^23 + j is exact in 32 bits, and so is its
    product with the scale, a power of two in base 2. The probabilities are then powers of two, at any size."""
    cache, tables, n, g = make_batch(lens, 16, nkv, D, cache_dtype, "NHD", seed=power)
    ks, vs = (0.5, 0.25) if cache_dtype == E4 else (1.0, 1.0)
    shape = cache.k.shape[:-1]
    k = torch.zeros(cache.k.shape, device=DEV)
    k[..., 0] = 256
    k[..., 1] = torch.randint(-3, 1, shape, generator=g, device=DEV)
    k = k.to(cache_dtype)
    cache = moe.MoeKvCache(k, cache.v, "NHD", ks, vs)
    nq = 6 * nkv
    q = torch.zeros((len(lens), nq, D), device=DEV, dtype=dtype)
    q[..., 0::2, 0], q[..., 1::2, 0] = 2.0 ** 15, -2.0 ** 15
    q[..., 1] = 1
    out, lse = torch.full_like(q, float("nan")), torch.full((len(lens), nq), float("nan"), device=DEV)
    scale = LN2 * 2.0 ** (power - 23) / ks
    moe.moe_attention_decode(q, cache, tables, n, out, scale, lse=lse)
    moe.moe_cache_check()
    u_o, u_p = {BF: 2.0 ** -8, FP: 2.0 ** -11}[dtype], 2.0 ** -8 if cache_dtype == BF else 2.0 ** -11
    for b, length in enumerate(lens):
        if length == 0:
            assert (out[b] == 0).all() and (lse[b] == float("-inf")).all()
            continue
        t = torch.arange(length, device=DEV)
        page, at = tables[b].long()[t // 16], t % 16
        rows = [x.view(torch.uint8)[page, at].contiguous().view(cache_dtype).float().double().transpose(0, 1) * s
                for x, s in ((k, ks), (cache.v, vs))]
        s = (q[b].double().view(nkv, 6, D) @ rows[0].transpose(1, 2)) * scale
        want = torch.logsumexp(s, -1, keepdim=True)
        p = torch.softmax(s, -1)   # not exp(s - want): 64 bits do not hold s and the logarithm of a count at 2^60
        o, size = p @ rows[1], p @ rows[1].abs()
        # scores differ by whole numbers times the scale, which is off by 2^-28 of its value from a power of two; p and
        # the output are rounded once each; 32-bit sums over the keys: n / 16 + 64 roundings, twice over; exp2 2^-21.
        # Scores above the largest by 128 steps of base 2 and more leave nothing, in 32 bits as in 64.
        rest = u_p + 2 * (length / 16 + 64) * 2.0 ** -24 + 2.0 ** -21 + 3 * 2.0 ** (min(power - 23, 8) - 28)
        assert ((out[b].double().view(nkv, 6, D) - o).abs() <= (size * rest + u_o * o.abs()) * 1.01 + 1e-30).all()
        # the logarithm: base plus log2 of the sum, and the product with ln 2: 4 roundings of its size
        off = (lse[b].double().view(nkv, 6, 1) - want).abs()
        assert (off <= 4 * 2.0 ** -24 * want.abs() + rest + 16 * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype,v_scale", [(BF, 2.0 ** -126), (BF, 1.7e-38), (BF, 2.0 ** -100), (BF, 2.0 ** 100), (FP, 2.0 ** -126),
                                           (FP, 2.0 ** -20), (FP, 64.0)])
@pytest.mark.parametrize("lens,nkv", [([1, 40, 700, 5000], 1), ([60000, 33], 2)])
def test_scales_of_values_at_the_ends_of_their_range(lens, nkv, v_scale, dtype):
    """Values of an 8-bit cache times a scale that is as small as a normal number may be, or large: outputs keep their
    relative accuracy wherever the output's type holds them (bf16: down to 2^-126)."""
    D, nq = 64, 6 * nkv
    cache, tables, n, g = make_batch(lens, 16, nkv, D, E4, "NHD", seed=len(lens))
    cache = moe.MoeKvCache(cache.k, cache.v, "NHD", 0.1, v_scale)
    q = normal((len(lens), nq, D), dtype, g, 1.0)
    out = torch.full_like(q, float("nan"))
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125)
    want, _, tol, _ = ref.attention(q, cache, tables, n, 0.125)
    assert want.abs().max() < (3e38 if dtype == BF else 65000)
    # below its normal numbers a type rounds by half a step of its smallest ones; the bound's own 1e-30 comes off
    tiny = 2.0 ** -134 if dtype == BF else 2.0 ** -25
    assert ((out.double() - want).abs() <= tol - 1e-30 * 1.01 + tiny).all()


@pytest.mark.parametrize("dtype,large,small,scale", [(BF, 2.0 ** 10, 2.0 ** -10, 2.0 ** 9), (BF, 2.0 ** 100, 2.0 ** 72, 2.0 ** -73), (FP, 60000.0, 2.0 ** -8, 2.0 ** 7),
                                                     (BF, 2.0 ** -110, 2.0 ** -126, 2.0 ** 125)])
@pytest.mark.parametrize("lens,nkv", [([1, 40, 700], 1), ([60000, 33], 2)])
def test_queries_of_very_different_elements_over_8_bits(lens, nkv, dtype, large, small, scale):
    """One element of q is 2^16 to 2^28 times the others and meets zeros: the scores come from the others alone, whose bits
    all count. fp16 queries are taken as they are. Of a bf16 head, whose largest element becomes 2^14 or more in fp16,
    an element is off by at most half a step of fp16's smallest numbers, 2^-25: 2^-39 of the largest."""
    D, nq = 64, 6 * nkv
    cache, tables, n, g = make_batch(lens, 16, nkv, D, E4, "NHD", seed=len(lens))
    cache.k.view(torch.uint8)[..., 5] = 0
    q = normal((len(lens), nq, D), torch.float32, g, 1.0).clamp(-3.9, 3.9) * small
    q = q.to(dtype)
    q[..., 5] = large
    out, lse = torch.full_like(q, float("nan")), torch.full((len(lens), nq), float("nan"), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, scale, lse=lse)
    if dtype == FP:
        check_attention(q, cache, tables, n, scale, 0, out, lse)
        return
    want, want_lse, tol, lse_tol = ref.attention(q, cache, tables, n, scale)
    size = ref.attention(q, moe.MoeKvCache(cache.k, (cache.v.view(torch.uint8) & 127).view(E4), "NHD", cache.k_scale, cache.v_scale),
                         tables, n, scale)[0]   # sum of p |v|
    for b, length in enumerate(lens):
        t = torch.arange(length, device=DEV)
        k = ref.cache_rows(cache, 0, "k", tables[b].long()[t // 16], t % 16).abs().sum(-1).amax(0)   # [nkv]
        moved = scale * 2.0 ** -39 * q[b].double().abs().amax(-1) * k.repeat_interleave(6)   # of each score
        # p moves by twice that (its score and the sum), the logarithm of the sum by as much
        assert ((out[b].double() - want[b]).abs() <= tol[b] + 2.02 * moved[:, None] * size[b]).all()
        assert ((lse[b].double() - want_lse[b]).abs() <= lse_tol[b] + moved).all()
