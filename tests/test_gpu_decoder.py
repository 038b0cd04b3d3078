"""The attention operators together, as a decoder uses them between its projections and the routed layer: prompts
of different lengths, single-token steps, a fork, an end and a compaction over one paged cache of two layers."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import moe_inputs as mi
import oracle
import mixture_experts_gemv_b200 as moe
from gpu_util import DevLayer, TOL_GEMV, ensure_init, rel_err
from mixture_experts_gemv_b200.paged_cache import PagedKvCache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_gemv_b200 import build
    build.build()
    yield
    moe.moe_cache_check()


class Decoder:
    """Two attention layers with random projections (torch's products) over the library's operators."""

    def __init__(self, d, nq, nkv, D, cache_dtype, window, layout, page):
        g = torch.Generator(device=DEV).manual_seed(7)
        self.d, self.nq, self.nkv, self.D, self.window = d, nq, nkv, D, window
        self.w_in = [torch.randn(d, (nq + 2 * nkv) * D, generator=g, device=DEV).mul_(d ** -0.5).to(BF) for _ in range(2)]
        self.w_out = [torch.randn(nq * D, d, generator=g, device=DEV).mul_((nq * D) ** -0.5).to(BF) for _ in range(2)]
        self.gains = [torch.rand(2, D, generator=g, device=DEV) + 0.5 for _ in range(2)]
        self.inv_freq, self.rope_scale = moe.moe_rope_frequencies(D // 2 // 16 * 16, 10000.0, moe.MOE_ROPE_YARN, 4.0, 64.0, device=DEV)
        scales = (0.05, 0.02) if cache_dtype == E4 else (1.0, 1.0)
        self.kv = PagedKvCache(2, 64, page, nkv, D, 6, 200, dtype=cache_dtype, layout=layout, k_scale=scales[0], v_scale=scales[1], device=DEV)

    def project(self, layer, x, positions, slots):
        T = x.shape[0]
        q, k, v = (x @ self.w_in[layer]).view(T, -1, self.D).split((self.nq, self.nkv, self.nkv), dim=1)
        out = torch.empty((T, self.nq, self.D), dtype=BF, device=DEV)
        moe.moe_qk_norm_rope(q, k, v, positions, self.inv_freq, q_gain=self.gains[layer][0], k_gain=self.gains[layer][1],
                             rope_scale=self.rope_scale, q_out=out, cache=self.kv.cache, layer=layer, slots=slots)
        want, size = ref.rotated(q, self.gains[layer][0], 1e-6, positions, self.inv_freq, False, self.rope_scale)
        assert ((out.double() - want).abs() <= ref.rotated_bound(want, size, self.D, BF)).all()
        return out

    def step(self, x, rows):
        """One token of each row (x [n, d]) through both layers; returns the last layer's output."""
        positions, slots = self.kv.append(rows, [1] * len(rows))
        at = torch.tensor(rows, device=DEV)
        for layer in range(2):
            q = self.project(layer, x, positions, slots)
            tables, lens = self.kv.block_tables[at], self.kv.seq_lens[at]
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
            moe.moe_attention_decode(q, self.kv.cache, tables, lens, out, self.D ** -0.5, window=self.window, layer=layer, lse=lse)
            want, want_lse, tol, lse_tol = ref.attention(q, self.kv.cache, tables, lens, self.D ** -0.5, self.window, layer)
            assert ((out.double() - want).abs() <= tol).all() and ((lse.double() - want_lse).abs() <= lse_tol).all()
            x = x + out.reshape(len(rows), -1) @ self.w_out[layer]
        return x


@pytest.mark.parametrize("cache_dtype,window,layout,page", [(BF, 0, "HND", 16), (E4, 0, "NHD", 8), (BF, 24, "NHD", 5)])
def test_decoding_over_one_cache(cache_dtype, window, layout, page):
    d, nq, nkv, D = 128, 8, 2, 64
    dec = Decoder(d, nq, nkv, D, cache_dtype, window, layout, page)
    g = torch.Generator(device=DEV).manual_seed(1)
    kv = dec.kv
    # prompts: keys and values of all their tokens, each layer's from inputs of its own (their attention is not the
    # single-token operator's)
    rows = [kv.open() for _ in range(3)]
    positions, slots = kv.append(rows, [33, 1, 50])
    for layer in range(2):
        dec.project(layer, torch.randn(84, d, generator=g, device=DEV).to(BF), positions, slots)
    x = torch.randn(3, d, generator=g, device=DEV).to(BF)
    for _ in range(12):
        x = dec.step(x, rows)
    # a fork goes on exactly as its parent does, page copies or not
    child = kv.fork(rows[0])
    x = torch.cat((x, x[:1]))
    for _ in range(2 * page + 1):
        x = dec.step(x, rows + [child])
        assert torch.equal(x[0], x[3])
    # one ends, its pages are given back and the others move up: the next step is the one it would have been
    kv.close(rows[1])
    left = [rows[0], rows[2], child]
    x = x[[0, 2, 3]]
    before = {kind: [ref.cache_rows(kv.cache, layer, kind, *places(kv, r)) for layer in range(2) for r in left] for kind in ("k", "v")}
    moved = kv.compact()
    assert moved > 0
    after = {kind: [ref.cache_rows(kv.cache, layer, kind, *places(kv, r)) for layer in range(2) for r in left] for kind in ("k", "v")}
    assert all(torch.equal(a, b) for kind in ("k", "v") for a, b in zip(before[kind], after[kind]))
    for _ in range(3):
        x = dec.step(x, left)
        assert torch.equal(x[0], x[2])
    moe.moe_cache_check()

    # the block's other half on the result: norm and routed layer, against the oracle
    E, f, k = 8, 64, 2
    lw = mi.make_layer(seed=3, d=d, f=f, E=E)
    dl = DevLayer(lw)
    ensure_init(3, d, f, E, k)
    moe.moe_set_path(moe.MOE_PATH_AUTO, 16)
    normed = torch.empty((3, d), dtype=BF, device=DEV)
    moe.moe_rmsnorm_bf16(x.float().contiguous(), normed, 3, d, 1e-6)
    out = torch.empty((3, d), dtype=torch.float32, device=DEV)
    moe.moe_layer_forward(normed, dl.router_w, dl.router_scale, dl.gate_up, dl.down, dl.expert_scale, 3, d, f, E, k, out)
    moe.moe_debug_check()
    bits = normed.view(torch.int16).cpu().numpy().view(np.uint16)
    want, _, _, flags = oracle.moe_layer(bits, lw.router_w, lw.router_scale, lw.gate_up, lw.down, lw.expert_scale, k)
    ok = (flags & 1) == 0
    assert ok.any() and rel_err(out.cpu().numpy()[ok], want[ok]) <= TOL_GEMV


def places(kv, row):
    at = torch.arange(kv.length(row), device=DEV)
    return kv.block_tables[row].long()[at // kv.page_size], at % kv.page_size


def test_a_captured_step_follows_the_tables_and_lengths():
    """Rotation, append and attention of one step as a graph: replayed while the sequences grow over page ends."""
    nq, nkv, D, page = 8, 2, 128, 16
    kv = PagedKvCache(1, 32, page, nkv, D, 4, 100, dtype=FP, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    inv, _ = moe.moe_rope_frequencies(D, device=DEV)
    rows = [kv.open() for _ in range(4)]
    positions, slots = kv.append(rows, [14, 1, 30, 15])
    new = lambda n: torch.randn(n, nq + 2 * nkv, D, generator=g, device=DEV).to(FP)  # noqa: E731
    q, k, v = new(60).split((nq, nkv, nkv), dim=1)
    moe.moe_qk_norm_rope(None, k, v, positions, inv, cache=kv.cache, slots=slots)
    qkv, pos, slot = new(4), torch.zeros(4, dtype=torch.int32, device=DEV), torch.full((4,), -1, dtype=torch.int64, device=DEV)
    turned, out = torch.empty((4, nq, D), dtype=FP, device=DEV), torch.empty((4, nq, D), dtype=FP, device=DEV)
    lse = torch.empty((4, nq), device=DEV)

    def one_step():
        q, k, v = qkv.split((nq, nkv, nkv), dim=1)
        moe.moe_qk_norm_rope(q, k, v, pos, inv, q_out=turned, cache=kv.cache, slots=slot)
        moe.moe_attention_decode(turned, kv.cache, kv.block_tables, kv.seq_lens, out, D ** -0.5, lse=lse)

    one_step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step()
    for i in range(20):
        counts = [1, 1, i % 2, 1]
        p, s = kv.append(rows, counts)
        slot.fill_(-1)
        at = torch.tensor([j for j, n in enumerate(counts) if n], device=DEV)
        pos[at], slot[at] = p, s
        qkv.copy_(new(4))
        graph.replay()
        want, want_lse, tol, lse_tol = ref.attention(turned, kv.cache, kv.block_tables, kv.seq_lens, D ** -0.5)
        assert ((out.double() - want).abs() <= tol).all() and ((lse.double() - want_lse).abs() <= lse_tol).all()
    moe.moe_cache_check()
