"""Norms and rotation with the append, one-token attention over a paged cache and page copies on the GPU, against
plain 64-bit forms, at the sizes, layouts, lengths and masks where they could go wrong."""
import os
import subprocess
import sys

import pytest
import torch

import attn_ref as ref
import mixture_experts_gemv_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_gemv_b200 import build
    build.build()
    yield
    moe.moe_cache_check()


def normal(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEV) * scale
    return x.clamp(-448, 448).to(dtype)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_cache(pages, page, nkv, D, dtype, layout, g, layers=None, poison=True):
    """A cache of NaN everywhere (what no call may let through), as two tensors."""
    shape = (pages, page, nkv, D) if layout == "NHD" else (pages, nkv, page, D)
    shape = shape if layers is None else (layers,) + shape
    fill = float("nan")
    k, v = (torch.full(shape, fill, device=DEV, dtype=torch.float32).to(dtype) for _ in range(2))
    scales = (0.11, 0.07) if dtype == E4 else (1.0, 1.0)
    return moe.MoeKvCache(k, v, layout, *scales)


def fill_rows(cache, page, off, g, layer=None):
    """Random rows at (page, off)."""
    for t in (cache.k, cache.v):
        t = t if layer is None else t[layer]
        spread = 12.0 if cache.dtype == E4 else 1.0
        rows = normal((len(page), cache.n_kv, cache.head_dim), cache.dtype, g, spread).view(torch.uint8)
        raw = t.view(torch.uint8)
        if cache.layout == "NHD":
            raw[page, off] = rows
        else:
            raw[page, :, off] = rows


def make_batch(lens, page, nkv, D, dtype, layout, seed, spare=2):
    """(cache, tables, lens): sequences over shuffled pages; everything outside them is NaN, unused entries -7."""
    g = gen(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    cache = make_cache(pages, page, nkv, D, dtype, layout, g)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        tables[b, : need[b]] = order[at: at + need[b]]
        at += need[b]
        if n > 0:
            t = torch.arange(n, device=DEV)
            fill_rows(cache, tables[b].long()[t // page], t % page, g)
    return cache, tables, torch.tensor(lens, dtype=torch.int32, device=DEV), g


def check_attention(q, cache, tables, lens, scale, window, out, lse, layer=0):
    want, want_lse, tol, lse_tol = ref.attention(q, cache, tables, lens, scale, window, layer)
    off = (out.double() - want).abs()
    assert (off <= tol).all(), f"out off by up to {float((off / tol.clamp(min=1e-300)).max()):.2f} of the bound"
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert ((lse.double() - want_lse).abs()[~empty] <= lse_tol[~empty]).all()
    assert (out[empty.any(-1)] == 0).all()


SHAPES = [  # n_q, n_kv, D, page, layout
    (1, 1, 16, 16, "NHD"), (4, 4, 64, 16, "HND"), (6, 2, 80, 5, "NHD"), (8, 1, 96, 24, "HND"), (16, 8, 128, 16, "NHD"),
    (18, 2, 128, 1, "NHD"), (40, 1, 128, 64, "HND"), (32, 2, 256, 16, "HND"), (24, 2, 240, 7, "NHD"),
    (8, 2, 512, 32, "NHD"), (20, 2, 400, 16, "HND"), (64, 1, 64, 128, "NHD"), (80, 1, 64, 16, "HND"),
    (30, 1, 48, 9, "NHD"),
]
LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 0, 700]


@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("nq,nkv,D,page,layout", SHAPES)
def test_attention_shapes(nq, nkv, D, page, layout, dtype, cache_dtype):
    cache, tables, lens, g = make_batch(LENS, page, nkv, D, cache_dtype, layout, seed=nq + D)
    q = normal((len(LENS), nq, D), dtype, g, 2.0)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((len(LENS), nq), float("nan"), device=DEV)
    scale = D ** -0.5
    moe.moe_attention_decode(q, cache, tables, lens, out, scale, lse=lse)
    check_attention(q, cache, tables, lens, scale, 0, out, lse)
    moe.moe_cache_check()


@pytest.mark.parametrize("window", [1, 16, 63, 64, 100, 10000])
@pytest.mark.parametrize("page,layout", [(16, "NHD"), (5, "HND")])
def test_attention_window(window, page, layout):
    lens = [0, 1, 15, 64, 65, 99, 100, 101, 128, 1000]
    cache, tables, n, g = make_batch(lens, page, 2, 64, BF, layout, seed=window)
    q = normal((len(lens), 6, 64), BF, g, 2.0)
    out, lse = torch.full_like(q, float("nan")), torch.empty((len(lens), 6), device=DEV)
    # pages wholly behind the window are not read: their entries name no page
    if window < 900:
        first = (1000 - window) // page
        tables[9, :first] = -7
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125, window=window, lse=lse)
    check_attention(q, cache, tables, n, 0.125, window, out, lse)
    moe.moe_cache_check()


@pytest.mark.parametrize("B,longest,nq,nkv,D,dtype,cache_dtype", [
    (1, 20011, 16, 2, 128, BF, BF), (1, 9001, 8, 1, 512, FP, FP), (300, 190, 8, 2, 64, BF, BF), (1, 30000, 32, 1, 256, BF, E4),
    (3, 8000, 8, 8, 256, BF, BF), (700, 40, 4, 4, 16, FP, FP)])
def test_attention_long_and_many(B, longest, nq, nkv, D, dtype, cache_dtype):
    """One long sequence cut over the whole grid; more sequences than a block has threads."""
    r = torch.Generator().manual_seed(B)
    lens = [longest] if B == 1 else torch.randint(0, longest, (B,), generator=r).tolist()
    cache, tables, n, g = make_batch(lens, 16, nkv, D, cache_dtype, "NHD", seed=B)
    q = normal((B, nq, D), dtype, g, 3.0)
    out, lse = torch.full_like(q, float("nan")), torch.empty((B, nq), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, D ** -0.5, lse=lse)
    check_attention(q, cache, tables, n, D ** -0.5, 0, out, lse)
    # the same bits again, and without lse
    again = torch.full_like(q, float("nan"))
    moe.moe_attention_decode(q, cache, tables, n, again, D ** -0.5)
    assert torch.equal(out, again)
    moe.moe_cache_check()


def test_attention_strided_rows_and_layers():
    """q and out are parts of wider rows, the cache's pages lie apart and its layers too; what is between stays."""
    lens, nq, nkv, D, page = [70, 3, 200], 12, 4, 64, 16
    g = gen(5)
    big = torch.full((3, 30, page, 2, nkv, D + 16), float("nan"), device=DEV, dtype=BF)
    k, v = big[:, :, :, 0, :, :D], big[:, :, :, 1, :, :D]
    cache = moe.MoeKvCache(k, v)
    tables = torch.full((3, 40), -7, dtype=torch.int32, device=DEV)[:, :15]
    for b, n in enumerate(lens):
        need = -(-n // page)
        tables[b, :need] = torch.arange(need, device=DEV, dtype=torch.int32) + 6 * b
        t = torch.arange(n, device=DEV)
        for x in (k, v):
            x[2][tables[b].long()[t // page], t % page] = normal((n, nkv, D), BF, g)
    wide = normal((3, nq + 5, D + 8), BF, g, 2.0)
    q = wide[:, 2: 2 + nq, :D]
    outw = torch.full((5, nq + 1, D + 24), 7.0, device=DEV, dtype=BF)
    out = outw[:3, :nq, :D]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lse = torch.empty((3, nq), device=DEV)
    before = wide.clone()
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125, layer=2, lse=lse)
    flat = moe.MoeKvCache(k[2], v[2])
    want, want_lse, tol, _ = ref.attention(q, flat, tables, n, 0.125)
    assert ((out.double() - want).abs() <= tol).all()
    left = outw.clone()
    left[:3, :nq, :D] = 7.0
    assert (left == 7.0).all() and torch.equal(wide, before)
    moe.moe_cache_check()


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 elements whose sequences lie at both of its ends."""
    page, nkv, D = 64, 8, 256
    pages = (1 << 32) // (page * nkv * D) + 40
    k = torch.empty((pages, page, nkv, D), dtype=E4, device=DEV)
    v = torch.empty_like(k)
    cache = moe.MoeKvCache(k, v, "NHD", 0.1, 0.05)
    tables = torch.tensor([[pages - 1, 3], [0, pages - 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([100, 128], dtype=torch.int32, device=DEV)
    g = gen(3)
    for b in range(2):
        t = torch.arange(128, device=DEV)
        fill_rows(cache, tables[b].long()[t // page], t % page, g)
    q = normal((2, 16, D), BF, g, 2.0)
    out, lse = torch.empty_like(q), torch.empty((2, 16), device=DEV)
    moe.moe_attention_decode(q, cache, tables, lens, out, 0.0625, lse=lse)
    check_attention(q, cache, tables, lens, 0.0625, 0, out, lse)
    # the append and the page copy reach the far end too
    new = normal((1, nkv, D), BF, g)
    slots = torch.tensor([(pages - 1) * page + 63], device=DEV)
    moe.moe_qk_norm_rope(None, new, new, None, None, cache=cache, slots=slots)
    got = ref.values(v[pages - 1, 63]) * 0.05
    assert ((got - new[0].double()).abs() <= ref.rotated_bound(new[0].double(), new[0].double().abs(), D, E4, 0.05)).all()
    moe.moe_copy_pages(cache, [pages - 1], [pages - 5])
    for t in (k, v):
        assert torch.equal(t[pages - 5].view(torch.uint8), t[pages - 1].view(torch.uint8))
    moe.moe_cache_check()


def test_attention_extreme_scores():
    """Scores far apart (one key takes all), equal scores, scores of -inf, and the type's largest values."""
    lens, D = [200, 200, 200, 40], 64
    cache, tables, n, g = make_batch(lens, 16, 1, D, FP, "NHD", seed=1)
    q = normal((4, 8, D), FP, g, 60.0)       # scores in the hundreds
    q[1] = 0                                   # all equal
    q[3] = 0
    q[3, :, 0] = 1.0
    kv = cache.k.view(-1, 1, D)
    rows = tables[3].long()[torch.arange(40, device=DEV) // 16] * 16 + torch.arange(40, device=DEV) % 16
    kv[rows, 0, 0] = float("-inf")            # every score -inf: no key is seen
    out, lse = torch.full_like(q, float("nan")), torch.empty((4, 8), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, 1.0, lse=lse)
    check_attention(q[:3], cache, tables[:3], n[:3], 1.0, 0, out[:3], lse[:3])
    assert (out[3] == 0).all() and (lse[3] == float("-inf")).all()
    # -inf on some keys only: as if they were not there
    kv[rows[20:], 0, 0] = 0.5
    moe.moe_attention_decode(q, cache, tables, n, out, 1.0, lse=lse)
    k = cache.k.view(-1, 1, D)[rows[20:], 0].double()
    v = cache.v.view(-1, 1, D)[rows[20:], 0].double()
    p = torch.softmax(q[3].double() @ k.T, -1)
    assert ((out[3].double() - p @ v).abs() <= (p @ v.abs()) * 2.0 ** -10 + 1e-6).all()
    # NaN and +inf inside a sequence reach its rows and no other's
    kv[rows[0], 0, 0] = float("nan")
    good = out[:3].clone()
    moe.moe_attention_decode(q, cache, tables, n, out, 1.0, lse=lse)
    assert torch.isnan(out[3]).all() and torch.equal(out[:3], good)


def test_attention_bf16_queries_beyond_fp16_over_8_bits():
    """bf16 queries above fp16's range (and below its smallest) over an e4m3 cache."""
    lens = [150, 150]
    cache, tables, n, g = make_batch(lens, 16, 2, 64, E4, "NHD", seed=9)
    q = normal((2, 4, 64), BF, g, 1.0)
    q[0] *= 2.0 ** 20
    q[1] *= 2.0 ** -30
    for b, scale in ((0, 2.0 ** -22), (1, 2.0 ** 28)):
        out, lse = torch.empty_like(q), torch.empty((2, 4), device=DEV)
        moe.moe_attention_decode(q, cache, tables, n, out, scale, lse=lse)
        s = slice(b, b + 1)
        check_attention(q[s], cache, tables[s], n[s], scale, 0, out[s], lse[s])


def test_attention_bad_pages_and_lengths_are_reported_and_not_followed():
    lens = [40, 40, 40]
    cache, tables, n, g = make_batch(lens, 16, 2, 64, BF, "NHD", seed=2)
    q = normal((3, 4, 64), BF, g)
    out, lse = torch.empty_like(q), torch.empty((3, 4), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125, lse=lse)
    moe.moe_cache_check()
    good = out.clone()
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        t = tables.clone()
        t[1, 1] = bad
        moe.moe_attention_decode(q, cache, t, n, out, 0.125, lse=lse)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_cache_check()
        assert e.value.code == moe.MOE_ERR_BAD_ARG and "block-table" in str(e.value)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and torch.isfinite(out[1]).all()
        moe.moe_cache_check()   # reported once
    for bad in (-5, 49, 2 ** 31 - 1):   # the table holds 48 tokens; past 40 lies NaN, in a page that exists
        m = n.clone()
        m[2] = bad
        moe.moe_attention_decode(q, cache, tables, m, out, 0.125, lse=lse)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_cache_check()
        assert "length" in str(e.value)
        assert torch.equal(out[:2], good[:2])


def test_attention_captured_and_replayed_with_other_inputs():
    lens = [300, 5, 64]
    cache, tables, n, g = make_batch(lens, 16, 2, 128, BF, "NHD", seed=4)
    q = normal((3, 16, 128), BF, g, 2.0)
    out, lse = torch.empty_like(q), torch.empty((3, 16), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, 0.1, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_attention_decode(q, cache, tables, n, out, 0.1, lse=lse)
    for step in range(3):
        n.copy_(torch.tensor([300 - 90 * step, step, 64 - step], dtype=torch.int32))
        q.copy_(normal((3, 16, 128), BF, g, 2.0))
        out.fill_(float("nan"))
        graph.replay()
        check_attention(q, cache, tables, n, 0.1, 0, out, lse)


def test_first_call_under_capture_in_a_new_process():
    code = """
import sys, torch
sys.path[:0] = [%r, %r]
import mixture_experts_gemv_b200 as moe
k = torch.randn(8, 16, 2, 64, device="cuda", dtype=torch.bfloat16); v = torch.randn_like(k)
cache = moe.MoeKvCache(k, v)
t = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
n = torch.tensor([60, 9], device="cuda", dtype=torch.int32)
q = torch.randn(2, 4, 64, device="cuda", dtype=torch.bfloat16); out = torch.zeros_like(q); qn = torch.zeros_like(q)
new = torch.randn(2, 2, 64, device="cuda", dtype=torch.bfloat16)
pos = torch.tensor([59, 8], device="cuda", dtype=torch.int32); slots = torch.tensor([59, 72], device="cuda")
f = moe.moe_rope_frequencies(64, device="cuda")[0]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_qk_norm_rope(q, new, new, pos, f, q_out=qn, cache=cache, slots=slots)
    moe.moe_attention_decode(qn, cache, t, n, out, 0.125)
    moe.moe_copy_pages(cache, [0], [7])
g.replay(); torch.cuda.synchronize()
want = out.clone(); out.zero_()
moe.moe_attention_decode(qn, cache, t, n, out, 0.125)
assert torch.equal(out, want) and out.abs().sum() > 0 and torch.equal(k[7], k[0])
moe.moe_cache_check()
print("fine")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_attention_calls_that_overlap_on_two_streams():
    """Each call has a workspace of its own: two streams at once give each call's own result."""
    work = []
    for seed, lens in ((1, [4000, 17]), (2, [1500, 2500])):
        cache, tables, n, g = make_batch(lens, 16, 4, 128, BF, "NHD", seed=seed)
        q = normal((2, 16, 128), BF, g, 2.0)
        out = torch.empty_like(q)
        moe.moe_attention_decode(q, cache, tables, n, out, 0.1)
        work.append((q, cache, tables, n, out.clone(), [torch.empty_like(q) for _ in range(20)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(20):
        for j, (q, cache, tables, n, _, outs, s) in enumerate(work):
            if j:
                with torch.cuda.stream(s):
                    moe.moe_attention_decode(q, cache, tables, n, outs[i], 0.1)
            else:
                moe.moe_attention_decode(q, cache, tables, n, outs[i], 0.1, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, want, outs, _ in work:
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("B,n_q,n_kv,longest", [(127, 4, 1, 600), (128, 4, 2, 400), (129, 8, 4, 300), (1300, 4, 2, 90), (5000, 2, 1, 40)])
@pytest.mark.parametrize("gap", [1, 5, 500])
def test_attention_many_sequences_with_empty_stretches(B, n_q, n_kv, longest, gap):
    """Batches around and past what a warp looks at together, most of them empty in long runs, the last among them."""
    r = torch.Generator().manual_seed(B + gap)
    lens = torch.randint(1, longest, (B,), generator=r)
    lens[(torch.arange(B) // gap) % 2 == 1] = 0
    lens[-3:] = 0
    cache, tables, n, g = make_batch(lens.tolist(), 16, n_kv, 64, BF, "NHD", seed=B)
    q = normal((B, n_q, 64), BF, g, 2.0)
    out, lse = torch.full_like(q, float("nan")), torch.empty((B, n_q), device=DEV)
    moe.moe_attention_decode(q, cache, tables, n, out, 0.125, lse=lse)
    check_attention(q, cache, tables, n, 0.125, 0, out, lse)
    moe.moe_cache_check()


@pytest.mark.parametrize("B,n_q,n_kv", [(64, 8, 1), (900, 8, 4)])
def test_attention_inputs_change_right_behind_a_call_that_cuts_no_sequence(B, n_q, n_kv):
    """Sequences of one unit each leave nothing to join: what follows still has to wait for the attention itself."""
    cache, tables, lens, g = make_batch([16] * B, 16, n_kv, 128, BF, "NHD", seed=B)
    q = normal((B, n_q, 128), BF, g, 2.0)
    out, lse = torch.empty_like(q), torch.empty((B, n_q), device=DEV)
    ql, ll, keep = q.clone(), lens.clone(), torch.empty_like(q)

    def step():
        ql.copy_(q)
        ll.copy_(lens)
        moe.moe_attention_decode(ql, cache, tables, ll, out, 0.1, lse=lse)
        keep.copy_(out)
        ll.zero_()
        ql.zero_()

    step()
    check_attention(q, cache, tables, lens, 0.1, 0, keep, lse)
    first = keep.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            step()
    for _ in range(20):
        keep.fill_(float("nan"))
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(keep, first)
    for _ in range(50):
        step()
        assert torch.equal(keep, first)
    moe.moe_cache_check()


def test_attention_given_workspace_holds_anything():
    lens = [777, 1]
    cache, tables, n, g = make_batch(lens, 16, 2, 256, FP, "HND", seed=6)
    q = normal((2, 4, 256), FP, g, 2.0)
    need = moe.moe_attention_decode_workspace_bytes(4, 2, 256)
    out, lse = torch.empty_like(q), torch.empty((2, 4), device=DEV)
    for fill in (0, 255):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=DEV)
        out.fill_(float("nan"))
        moe.moe_attention_decode(q, cache, tables, n, out, 0.0625, lse=lse, workspace=ws[:need])
        check_attention(q, cache, tables, n, 0.0625, 0, out, lse)
        assert (ws[need:] == fill).all()


# ------------------------------------------------------------------ norms, rotation, append

ROPE = [  # T, n_q, n_kv, D, rotary_dim, interleaved, norm, far
    (1, 16, 8, 128, 128, False, True, 0), (8, 16, 8, 256, 256, False, True, 9000), (3, 1, 1, 16, 16, False, True, 5),
    (5, 3, 1, 96, 96, False, True, 77), (130, 6, 2, 80, 32, False, True, 262000), (257, 4, 4, 64, 64, True, True, 100),
    (33, 2, 1, 512, 128, True, False, 240000), (19, 5, 5, 48, 6, True, True, 2 ** 30), (7, 8, 2, 400, 0, False, True, 0),
    (2500, 8, 2, 128, 64, False, True, 0), (64, 40, 1, 240, 240, True, True, 10), (12, 7, 3, 512, 512, False, True, 1),
    (11, 4, 2, 112, 98, True, True, 3000),
]


@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("T,nq,nkv,D,rot,inter,norm,far", ROPE)
def test_norm_rope_and_append(T, nq, nkv, D, rot, inter, norm, far, dtype, cache_dtype):
    g = gen(T + D)
    page, layout = (16, "NHD") if T % 2 else (5, "HND")
    qkv = normal((T, nq + 2 * nkv, D), dtype, g, 1.5)
    q, k, v = qkv.split((nq, nkv, nkv), dim=1)
    pos = (torch.arange(T, device=DEV) + far).to(torch.int32)
    inv = moe.moe_rope_frequencies(rot, 10000.0, device=DEV)[0] if rot else None
    qg, kg = (torch.randn(D, generator=g, device=DEV) for _ in range(2)) if norm else (None, None)
    cache = make_cache(-(-T // page) + 2, page, nkv, D, cache_dtype, layout, g)
    slots = torch.randperm(cache.num_pages * page, generator=g, device=DEV)[:T]
    if T > 4:
        slots[T // 2] = -1
    q_out = torch.full((T, nq, D), float("nan"), device=DEV, dtype=dtype)
    k_out = torch.full((T, nkv, D), float("nan"), device=DEV, dtype=dtype)
    before = qkv.clone()
    moe.moe_qk_norm_rope(q, k, v, pos, inv, q_gain=qg, k_gain=kg, interleaved=inter, rope_scale=1.25, q_out=q_out, k_out=k_out,
                         cache=cache, slots=slots)
    moe.moe_cache_check()
    assert torch.equal(qkv, before)
    yq, size = ref.rotated(q, qg, 1e-6, pos, inv, inter, 1.25)
    assert ((q_out.double() - yq).abs() <= ref.rotated_bound(yq, size, D, dtype)).all()
    yk, size = ref.rotated(k, kg, 1e-6, pos, inv, inter, 1.25)
    assert ((k_out.double() - yk).abs() <= ref.rotated_bound(yk, size, D, dtype)).all()
    ks, vs = cache.k_scale, cache.v_scale
    ok = slots >= 0
    at = slots[ok]
    got = ref.cache_rows(cache, 0, "k", at // page, at % page)
    lim = 448 * ks if cache_dtype == E4 else float("inf")
    want = yk[ok].clamp(-lim, lim)
    assert ((got - want).abs() <= ref.rotated_bound(want, size[ok], D, cache_dtype, ks)).all()
    got = ref.cache_rows(cache, 0, "v", at // page, at % page)
    want = v[ok].double()
    if cache_dtype == E4:
        assert ((got - want).abs() <= ref.rotated_bound(want, want.abs(), D, E4, vs)).all()
    else:
        assert torch.equal(got, want)
    # every other row of the cache is as it was
    other = torch.ones(cache.num_pages * page, dtype=torch.bool, device=DEV)
    other[at] = False
    rest = other.nonzero()[:, 0]
    for kind in ("k", "v"):
        assert torch.isnan(ref.cache_rows(cache, 0, kind, rest // page, rest % page)).all()


def test_rope_in_place_and_outputs_alone():
    g = gen(8)
    T, nq, nkv, D = 37, 8, 2, 128
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    inv, _ = moe.moe_rope_frequencies(D, device=DEV)
    gain = torch.randn(D, generator=g, device=DEV)
    qkv = normal((T, nq + 2 * nkv, D), BF, g)
    q, k, v = qkv.split((nq, nkv, nkv), dim=1)
    qo, ko = torch.empty((T, nq, D), device=DEV, dtype=BF), torch.empty((T, nkv, D), device=DEV, dtype=BF)
    moe.moe_qk_norm_rope(q, k, None, pos, inv, q_gain=gain, k_gain=gain, q_out=qo, k_out=ko)
    q_only, k_only = torch.empty_like(qo), torch.empty_like(ko)
    moe.moe_qk_norm_rope(q, None, None, pos, inv, q_gain=gain, q_out=q_only)
    moe.moe_qk_norm_rope(None, k, None, pos, inv, k_gain=gain, k_out=k_only)
    assert torch.equal(qo, q_only) and torch.equal(ko, k_only)
    v0 = v.clone()
    moe.moe_qk_norm_rope(q, k, v, pos, inv, q_gain=gain, k_gain=gain, q_out=q, k_out=k)   # parts of one buffer, in place
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, v0)


@pytest.mark.parametrize("cache_dtype", [BF, E4])
def test_rope_heads_and_tokens_apart(cache_dtype):
    """Heads that are not neighbours, wide tokens, more heads than one block takes; what is between stays."""
    g = gen(12)
    T, nq, nkv, D = 21, 70, 9, 96
    wide = normal((T, nq + 2 * nkv + 3, D + 16), BF, g)
    q, k, v = wide[:, 1: 1 + nq, :D], wide[:, nq + 1: nq + 1 + nkv, :D], wide[:, nq + nkv + 2: nq + 2 * nkv + 2, 16:]
    outs = torch.full((T, nq + nkv + 1, D + 8), 7.0, device=DEV, dtype=BF)
    q_out, k_out = outs[:, :nq, :D], outs[:, nq + 1:, :D]
    pos = torch.arange(T, device=DEV, dtype=torch.int32) * 11
    inv, _ = moe.moe_rope_frequencies(64, device=DEV)
    qg, kg = (torch.randn(D, generator=g, device=DEV) for _ in range(2))
    kv = torch.zeros((2, 5, 9, nkv + 2, D + 32), device=DEV, dtype=torch.float32).to(cache_dtype)
    cache = moe.MoeKvCache(kv[0, :, 1:6, :nkv, 16: 16 + D], kv[1, :, 1:6, :nkv, 16: 16 + D], "NHD",
                           *((0.05, 0.04) if cache_dtype == E4 else (1.0, 1.0)))
    slots = torch.randperm(25, generator=g, device=DEV)[:T]
    before = wide.clone()
    moe.moe_qk_norm_rope(q, k, v, pos, inv, q_gain=qg, k_gain=kg, q_out=q_out, k_out=k_out, cache=cache, slots=slots)
    moe.moe_cache_check()
    assert torch.equal(wide, before)
    for x, gain, out in ((q, qg, q_out), (k, kg, k_out)):
        want, size = ref.rotated(x, gain, 1e-6, pos, inv, False)
        assert ((out.double() - want).abs() <= ref.rotated_bound(want, size, D, BF)).all()
    want, size = ref.rotated(k, kg, 1e-6, pos, inv, False)
    got = ref.cache_rows(cache, 0, "k", slots // 5, slots % 5)
    assert ((got - want).abs() <= ref.rotated_bound(want, size, D, cache_dtype, cache.k_scale)).all()
    got = ref.cache_rows(cache, 0, "v", slots // 5, slots % 5)
    assert ((got - v.double()).abs() <= ref.rotated_bound(v.double(), v.double().abs(), D, cache_dtype, cache.v_scale)).all()
    left = outs.clone()
    left[:, :nq, :D] = 7.0
    left[:, nq + 1:, :D] = 7.0
    assert (left == 7.0).all()
    raw = kv.view(torch.uint8)
    es = 1 if cache_dtype == E4 else 2
    held = torch.zeros(raw.shape, dtype=torch.bool, device=DEV)
    for i in range(2):
        part = held[i, :, 1:6, :nkv, 16 * es: (16 + D) * es]
        part[slots // 5, slots % 5] = True
    assert (raw[~held] == 0).all()


def test_rope_infinities_stay_in_their_pairs():
    """Without a norm an infinity reaches its rotation partner alone, and none beyond rotary_dim."""
    for inter in (False, True):
        x = torch.ones((1, 1, 64), device=DEV, dtype=BF)
        x[0, 0, 3] = float("inf")
        x[0, 0, 40] = float("inf")   # past rotary_dim
        out = torch.empty_like(x)
        moe.moe_qk_norm_rope(x, None, None, torch.tensor([1], device=DEV, dtype=torch.int32),
                             moe.moe_rope_frequencies(32, device=DEV)[0], interleaved=inter, q_out=out)
        bad = (~torch.isfinite(out[0, 0])).nonzero()[:, 0].tolist()
        assert bad == ([2, 3, 40] if inter else [3, 19, 40])
        assert out[0, 0, 40] == float("inf")


def test_rope_bad_slots_are_reported_and_not_written():
    g = gen(9)
    cache = make_cache(4, 16, 2, 64, BF, "NHD", g)
    k = normal((3, 2, 64), BF, g)
    for bad in (64, 2 ** 40):
        slots = torch.tensor([5, bad, -3], device=DEV)
        moe.moe_qk_norm_rope(None, k, k, None, None, cache=cache, slots=slots)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_cache_check()
        assert "slot" in str(e.value)
        assert torch.equal(cache.v[0, 5], k[0])
        assert torch.isnan(cache.k.float()).sum() == 63 * 2 * 64


# ------------------------------------------------------------------ page copies

@pytest.mark.parametrize("layout", ["NHD", "HND", "gaps", "planes"])
@pytest.mark.parametrize("dtype,page,nkv,D,layers", [(BF, 16, 8, 128, 3), (E4, 5, 1, 48, 2), (FP, 1, 3, 16, 1), (E4, 128, 2, 512, 2)])
def test_copy_pages_and_tables(layout, dtype, page, nkv, D, layers):
    g = gen(page)
    pages = 60
    shape = {"NHD": (layers, pages, page, nkv, D), "HND": (layers, pages, nkv, page, D),
             "gaps": (layers, pages, page + 1, nkv + 1, D + 16), "planes": (nkv, layers, pages, page, D)}[layout]
    bits = [torch.randint(0, 256, shape[:-1] + (shape[-1] * torch.empty(0, dtype=dtype).element_size(),), generator=g,
                          device=DEV, dtype=torch.uint8) for _ in range(2)]
    k, v = (b.view(dtype) for b in bits)
    if layout == "gaps":
        k, v = (t[:, :, :page, :nkv, :D] for t in (k, v))
    if layout == "planes":   # each KV head's pages apart
        k, v = (t.permute(1, 2, 0, 3, 4) for t in (k, v))
    cache = moe.MoeKvCache(k, v, "HND" if layout in ("HND", "planes") else "NHD")
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    src, dst = order[:17], order[17:34]
    tables = torch.randint(-1, pages, (6, 9), generator=g, device=DEV, dtype=torch.int32)[:, :7]
    want_bits = [b.clone() for b in bits]
    for b, t in zip(want_bits, (k, v)):
        w = torch.as_strided(b.view(dtype), t.shape, t.stride(), 0)
        w8 = w.view(torch.uint8)
        w8[:, dst.long().to(DEV)] = w8[:, src.long().to(DEV)]
    to = {int(a): int(b) for a, b in zip(src, dst)}
    want_t = torch.tensor([[to.get(e, e) for e in row] for row in tables.tolist()], dtype=torch.int32, device=DEV)
    moe.moe_copy_pages(cache, src, dst, block_tables=tables)
    assert all(torch.equal(a, b) for a, b in zip(bits, want_bits))
    assert torch.equal(tables, want_t)
    # a fork: one source, several destinations, no table
    moe.moe_copy_pages(cache, [int(src[0])] * 3, dst[:3].tolist())
    raw = cache.k.view(torch.uint8)
    for d in dst[:3].tolist():
        assert torch.equal(raw[:, d], raw[:, int(src[0])])
    moe.moe_copy_pages(cache, [], [])


def test_copy_pages_longer_than_one_launch_holds():
    pages = 9000
    k = torch.arange(pages, device=DEV, dtype=torch.int32).view(pages, 1, 1, 1).expand(pages, 1, 1, 16).contiguous().view(BF)
    k = k.view(pages, 1, 1, 32).clone()
    v = k.clone()
    cache = moe.MoeKvCache(k, v)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    src, dst = order[:4400], order[4400:8800]
    tables = torch.arange(pages, device=DEV, dtype=torch.int32).view(30, 300)
    want = k.clone()
    want[dst.long().to(DEV)] = k[src.long().to(DEV)]
    moe.moe_copy_pages(cache, src, dst, block_tables=tables)
    assert torch.equal(k.view(torch.int16), want.view(torch.int16)) and torch.equal(v.view(torch.int16), want.view(torch.int16))
    to = torch.arange(pages, dtype=torch.int32)
    to[src.long()] = dst
    assert torch.equal(tables.cpu().view(-1), to)
