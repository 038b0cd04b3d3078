"""The attention entry points without a GPU: what they refuse before touching the device, and the host function
of the rotation's frequencies."""
import ctypes
import math

import pytest
import torch

import mixture_experts_gemv_b200 as moe
from mixture_experts_gemv_b200._lib import _HEADS, _KV_CACHE

FAKE = 1 << 20   # an aligned address that nothing here follows


@pytest.fixture(scope="module")
def L():
    from mixture_experts_gemv_b200 import build
    build.build()
    return moe.lib()


def kv(**change):
    a = dict(k=FAKE, v=FAKE + (1 << 30), dtype=moe.MOE_DT_BF16, n_layers=2, num_pages=50, page_size=16, n_kv=2, head_dim=64,
             layer_stride=50 * 2048, page_stride=2048, token_stride=128, head_stride=64, k_scale=1.0, v_scale=1.0)
    a.update(change)
    a["k"] = a["k"] or 0
    return _KV_CACHE.pack(*a.values())


def heads(at=FAKE, token=512, head=64):
    return _HEADS.pack(at or 0, token, head)


def code(L, rc, want, text=""):
    assert rc == want, L.moe_last_error()
    assert text in L.moe_last_error().decode()


BAD_CACHES = [
    (dict(k=None), -2), (dict(dtype=3), -2), (dict(head_dim=24), -2), (dict(head_dim=528), -2), (dict(head_dim=0), -2),
    (dict(num_pages=0), -2), (dict(page_size=0), -2), (dict(n_kv=0), -2), (dict(n_layers=0), -2),
    (dict(k=FAKE + 8), -3), (dict(token_stride=132), -3), (dict(head_stride=60), -3), (dict(page_stride=-2048), -2),
    (dict(token_stride=64), -2),        # tokens on top of heads
    (dict(page_stride=1024), -2), (dict(layer_stride=2048), -2), (dict(head_stride=0), -2),
    (dict(k_scale=0.5), -2), (dict(dtype=moe.MOE_DT_E4M3, v_scale=0.0), -2), (dict(dtype=moe.MOE_DT_E4M3, k_scale=float("inf")), -2),
    (dict(dtype=moe.MOE_DT_E4M3, k_scale=float("nan")), -2), (dict(dtype=moe.MOE_DT_E4M3, v_scale=1e-39), -2), (dict(dtype=moe.MOE_DT_E4M3, k_scale=-1.0), -2),
]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(L, change, want):
    c, h, o = kv(**change), heads(), heads(FAKE * 8)
    dt = moe.MOE_DT_BF16
    ws = L.moe_attention_decode_workspace_bytes(4, 2, 64)
    assert L.moe_attention_decode(h, dt, c, 0, FAKE, 4, 4, FAKE, 1, 4, 1.0, 0, o, None, FAKE, ws, None) == want
    one = (ctypes.c_int32 * 1)(1)
    two = (ctypes.c_int32 * 1)(2)
    assert L.moe_copy_pages(c, one, two, 1, None, 0, 0, 0, None) == want
    hd = change.get("head_dim", 64)
    rc = L.moe_qk_norm_rope(None, heads(), heads(FAKE * 4), dt, 1, 0, 2, 64, None, None, 0, 0, 1.0, None, None, 0.0, None, None, c, 0,
                            FAKE, None)
    assert rc == want or hd != 64


def attn(L, q=None, dt=0, c=None, layer=0, tables=FAKE, stride=4, cols=4, lens=FAKE, B=1, nq=4, scale=1.0, window=0, out=None,
         ws=FAKE, size=None):
    c = kv() if c is None else c
    size = L.moe_attention_decode_workspace_bytes(4, 2, 64) if size is None else size
    return L.moe_attention_decode(heads() if q is None else q, dt, c, layer, tables, stride, cols, lens, B, nq, scale, window,
                                  heads(FAKE * 8) if out is None else out, None, ws, size, None)


def test_attention_refusals(L):
    for a in (dict(dt=2), dict(dt=7), dict(dt=1), dict(layer=2), dict(layer=-1), dict(tables=None), dict(lens=None), dict(ws=None),
              dict(stride=3), dict(cols=0), dict(B=-1), dict(nq=3), dict(nq=0), dict(nq=8192), dict(B=2**30 + 1), dict(window=-1), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(scale=3e38), dict(size=100), dict(cols=1 << 27, stride=1 << 27), dict(q=heads(None)), dict(q=heads(token=-8)),
              dict(out=heads(FAKE * 8, 256, 32)), dict(B=3, out=heads(FAKE * 8, 64, 64)), dict(out=heads(FAKE + 256)), dict(out=heads())):
        assert attn(L, **a) == -2, a
        assert L.moe_last_error()
    for a in (dict(q=heads(FAKE + 2)), dict(q=heads(head=68)), dict(out=heads(FAKE * 8, 516)), dict(ws=FAKE + 8)):
        assert attn(L, **a) == -3, a
    assert attn(L, B=0) == 0
    for a in (dict(tables=FAKE + 2), dict(lens=FAKE + 1)):
        assert attn(L, **a) == -3, a
    # out may lie between q's heads and tokens of one buffer, not on them
    assert attn(L, B=0, q=heads(FAKE, 1024, 64), out=heads(FAKE + 512, 1024, 64)) == 0
    assert attn(L, B=3, q=heads(FAKE, 1024, 64), out=heads(FAKE + 504 + 4, 1024, 64)) == -3
    assert attn(L, B=3, q=heads(FAKE, 1024, 64), out=heads(FAKE + 496, 1024, 64)) == -2
    assert L.moe_attention_decode_workspace_bytes(5, 2, 64) == 0
    assert L.moe_attention_decode_workspace_bytes(4, 2, 65) == 0
    assert L.moe_attention_decode_workspace_bytes(8192, 2, 64) == 0
    assert L.moe_attention_decode_workspace_bytes(4, 0, 64) == 0


def rope(L, q=True, k=True, v=True, dt=0, T=3, nq=4, nkv=2, D=64, pos=FAKE, inv=FAKE, rot=64, inter=0, scale=1.0, qg=None, kg=None, eps=1e-6,
         qo=True, ko=True, c=None, layer=0, slots=FAKE):
    at = [heads(FAKE * (2 * i + 1)) for i in range(5)]
    pick = lambda x, i: at[i] if x is True else x  # noqa: E731
    return L.moe_qk_norm_rope(pick(q, 0), pick(k, 1), pick(v, 2), dt, T, nq, nkv, D, pos, inv, rot, inter, scale, qg, kg, eps, pick(qo, 3),
                              pick(ko, 4), c, layer, slots, None)


def test_norm_rope_refusals(L):
    c = kv(k=FAKE * 64, v=FAKE * 2048)
    for a in (dict(dt=2), dict(T=-1), dict(nq=-1), dict(nq=0, nkv=0), dict(D=40), dict(D=1024), dict(rot=24), dict(rot=128), dict(rot=-2),
              dict(rot=33, inter=1), dict(pos=None), dict(inv=None), dict(scale=float("nan")), dict(eps=-1.0), dict(eps=float("nan")),
              dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(c=c, v=None), dict(c=c, slots=None), dict(c=c, nkv=0),
              dict(c=c, layer=2), dict(c=c, nkv=1), dict(c=c, D=48, rot=48), dict(c=kv(dtype=1)), dict(qo=heads(FAKE * 7, 512, 32)),
              dict(qo=heads(FAKE * 7, 128, 64)), dict(qo=heads(FAKE, 512, 128)), dict(qo=heads(FAKE + 128)), dict(ko=heads(FAKE * 7)),
              dict(qo=heads(FAKE * 3)), dict(c=c, qo=heads(FAKE * 5)), dict(qo=heads(FAKE * 3 - 256))):
        assert rope(L, **a) == -2, a
    assert rope(L, c=kv(k=FAKE * 64, v=FAKE * 64)) == -2
    for a in (dict(q=heads(FAKE + 8)), dict(pos=FAKE + 2), dict(inv=FAKE + 4), dict(c=c, slots=FAKE + 4), dict(qg=FAKE + 4), dict(kg=FAKE + 8), dict(ko=heads(FAKE * 9, 516)), dict(c=kv(v=FAKE + 2))):
        assert rope(L, **a) == -3, a
    assert rope(L, T=0) == 0
    # q and k as parts of one buffer's rows may be turned in place; a part that reaches into the next may not
    q, k = heads(FAKE, 512, 64), heads(FAKE + 4 * 64 * 2, 512, 64)
    assert rope(L, q=q, k=k, qo=q, ko=k, T=0) == 0
    assert rope(L, q=q, k=k, nq=5, qo=q, ko=k) == -2


def pages(L, src, dst, c=None, tables=None, stride=4, rows=2, cols=4):
    n = len(src)
    a = (ctypes.c_int32 * max(n, 1))(*src)
    b = (ctypes.c_int32 * max(n, 1))(*dst)
    return L.moe_copy_pages(kv() if c is None else c, a, b, n, tables, stride, rows, cols, None)


def test_copy_pages_refusals(L):
    for src, dst in (([50], [1]), ([1], [50]), ([-1], [1]), ([1], [-1]), ([1], [1]), ([1, 2], [2, 3]), ([1, 2], [3, 3]), ([2, 1], [3, 2]),
                     (list(range(50)) + [0], [49] * 51)):
        code(L, pages(L, src, dst), -2, "page" if len(src) < 50 else "pages")
    code(L, pages(L, [1, 1], [2, 3], tables=FAKE), -2, "moves twice")
    code(L, pages(L, [1], [2], tables=FAKE + 2), -3)
    code(L, pages(L, [1], [2], tables=FAKE, stride=3), -2)
    code(L, pages(L, [1], [2], tables=FAKE, rows=-1), -2)
    assert pages(L, [], []) == 0
    assert L.moe_copy_pages(kv(), None, None, 1, None, 0, 0, 0, None) == -2
    assert L.moe_copy_pages(kv(), None, None, -1, None, 0, 0, 0, None) == -2
    assert L.moe_copy_pages(None, None, None, 0, None, 0, 0, 0, None) == -2


def test_good_calls_without_a_gpu_fail_cleanly(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert attn(L) in (-4, -6)
    assert rope(L) in (-4, -6)
    assert pages(L, [1], [2]) in (-4, -6)
    assert L.moe_cache_check(None) in (-4, -6)


def test_binding_refuses_what_the_library_cannot_see():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    bad = moe.MoeError
    for a in ((k, k[:2]), (k, k.half()), (k.float(), k.float()), (k[0], k[0]), (k[..., ::2], k[..., ::2])):
        with pytest.raises(bad):
            moe.MoeKvCache(*a)
    with pytest.raises(bad):
        moe.MoeKvCache(k, k.clone(), "DHN")
    cache = moe.MoeKvCache(k, k.clone())
    q, out = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(q=q, cache=cache, block_tables=t, seq_lens=n, out=out, scale=1.0)
    for a in (dict(q=q[0]), dict(q=q[..., :32]), dict(out=out[:1]), dict(out=out.half()), dict(block_tables=t[:1]), dict(block_tables=t.long()),
              dict(block_tables=t.t().contiguous().t()), dict(seq_lens=n.long()), dict(seq_lens=n[:1]), dict(lse=torch.zeros(2, 4).double()),
              dict(lse=torch.zeros(4, 2).t()), dict(q=q.float()), dict()):   # the last: not on a GPU
        with pytest.raises(bad):
            moe.moe_attention_decode(**{**good, **a})
    f = torch.zeros(32, dtype=torch.float64)
    pos = torch.zeros(2, dtype=torch.int32)
    good = dict(q=q, k=None, v=None, positions=pos, inv_freq=f, q_out=out)
    for a in (dict(q=None), dict(positions=None), dict(positions=pos.long()), dict(inv_freq=f.float()), dict(q_out=out[:1]),
              dict(q_gain=torch.zeros(32)), dict(cache=cache, k=q[:, :2], v=q[:, :2]), dict(k=q[:1]),
              dict(cache=cache, k=q[:, :2], v=q[:, :2], slots=pos), dict()):
        with pytest.raises(bad):
            moe.moe_qk_norm_rope(**{**good, **a})
    for src, dst in (([1], [2, 3]), (torch.tensor([1]), torch.tensor([2], dtype=torch.int32)), ([1], [2])):
        with pytest.raises(bad):
            moe.moe_copy_pages(cache, src, dst)


def test_one_cache_descriptor_for_both_orders_and_layers():
    nhd = torch.zeros(3, 7, 16, 2, 64, dtype=torch.float8_e4m3fn)
    a = moe.MoeKvCache(nhd, nhd.clone(), "NHD", 0.5, 0.25)
    assert _KV_CACHE.unpack(a.packed)[2:] == (moe.MOE_DT_E4M3, 3, 7, 16, 2, 64, 7 * 2048, 2048, 128, 64, 0.5, 0.25)
    hnd = torch.zeros(7, 2, 16, 64, dtype=torch.float16)
    b = moe.MoeKvCache(hnd, hnd.clone(), "HND")
    assert _KV_CACHE.unpack(b.packed)[2:] == (moe.MOE_DT_F16, 1, 7, 16, 2, 64, 0, 2048, 64, 1024, 1.0, 1.0)
    assert (b.n_layers, b.num_pages, b.page_size, b.n_kv, b.head_dim) == (1, 7, 16, 2, 64)


def test_frequencies():
    for rot in (2, 64, 98):
        f, s = moe.moe_rope_frequencies(rot, 10000.0)
        want = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
        assert s == 1.0 and max(abs(a / b - 1) for a, b in zip(f.tolist(), want)) < 1e-14
    plain = moe.moe_rope_frequencies(64, 500000.0)[0]
    assert torch.allclose(moe.moe_rope_frequencies(64, 500000.0, moe.MOE_ROPE_LINEAR, 8.0)[0], plain / 8, rtol=1e-14, atol=0)
    ntk = moe.moe_rope_frequencies(64, 10000.0, moe.MOE_ROPE_NTK, 8.0)[0]
    # the scaled base leaves the fastest pair alone and slows the slowest by the factor
    p = moe.moe_rope_frequencies(64, 10000.0)[0]
    assert ntk[0] == p[0] and abs(float(ntk[-1] / p[-1]) * 8 - 1) < 1e-12
    # a factor of 1 changes nothing, whichever kind
    for kind in (moe.MOE_ROPE_LINEAR, moe.MOE_ROPE_NTK, moe.MOE_ROPE_YARN):
        f, s = moe.moe_rope_frequencies(64, 10000.0, kind, 1.0)
        assert torch.equal(f, p) and s == 1.0


def test_yarn_frequencies_keep_fast_pairs_and_interpolate_slow_ones():
    rot, base, factor, length, fast, slow = 128, 10000.0, 16.0, 4096.0, 32.0, 1.0
    f, s = moe.moe_rope_frequencies(rot, base, moe.MOE_ROPE_YARN, factor, length, fast, slow)
    p = moe.moe_rope_frequencies(rot, base)[0]
    assert abs(s - (0.1 * math.log(factor) + 1)) < 1e-6
    turns = p * length / (2 * math.pi)
    at = lambda b: rot * math.log(length / (b * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(at(fast)), math.ceil(at(slow))
    for i in range(rot // 2):
        if i <= lo:
            assert f[i] == p[i] and turns[i] >= fast * 0.99
        elif i >= hi:
            assert abs(float(f[i] * factor / p[i]) - 1) < 1e-14 and turns[i] <= slow * 1.01
        else:
            share = (i - lo) / (hi - lo)
            assert abs(float(f[i] / (p[i] * (share / factor + 1 - share))) - 1) < 1e-12
    assert (f[1:] < f[:-1]).all()


@pytest.mark.parametrize("a", [dict(kind=4), dict(kind=-1), dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=514), dict(base=1.0),
                               dict(base=float("nan")), dict(factor=0.5), dict(factor=float("inf")), dict(kind=2, rotary_dim=2),
                               dict(kind=3, original_length=0.0), dict(kind=3, beta_slow=0.0), dict(kind=3, beta_fast=1.0)])
def test_frequency_refusals(a):
    with pytest.raises(moe.MoeError):
        moe.moe_rope_frequencies(**{**dict(rotary_dim=64, factor=2.0), **a})
