"""Which rows of q, k, v and outputs may lie in one buffer: what the entry points refuse, against sets of addresses. (The
calls that are accepted would follow their made-up addresses on a GPU: these run where there is none.)"""
import random

import pytest
import torch

import mixture_experts_gemv_b200 as moe
from mixture_experts_gemv_b200._lib import _HEADS, _KV_CACHE

FAKE = 1 << 30


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    from mixture_experts_gemv_b200 import build
    build.build()
    return moe.lib()


def places(at, token, head, T, n, D):
    return {at + t * token + h * head + i for t in range(T) for h in range(n) for i in range(0, D, 8)}


def heads(at, token, head):
    return _HEADS.pack(FAKE + 2 * at, token, head)


def rope(L, T, nq, nkv, D, q, k, q_out, k_out):
    return L.moe_qk_norm_rope(heads(*q), heads(*k), None, 0, T, nq, nkv, D, None, None, 0, 0, 1.0, None, None, 0.0, heads(*q_out),
                              heads(*k_out), None, 0, None, None)


def layouts(r, n, D, token):
    """(at, token stride, head stride) of n heads in tokens `token` apart."""
    head = r.choice((D, 2 * D, 3 * D, D + 8))
    return 8 * r.randrange(0, 40), token, head


def test_refusals_against_sets_of_addresses(L):
    r = random.Random(5)
    accepted = refused = 0
    while accepted < 400 or refused < 400:
        T, nq, nkv, D = r.randrange(1, 4), r.randrange(1, 4), r.randrange(1, 4), 16
        token = 8 * r.randrange(2, 60)
        tokens = [token if r.random() < 0.9 else 8 * r.randrange(2, 60) for _ in range(4)]
        q, k, q_out, k_out = (layouts(r, n, D, t) for n, t in zip((nq, nkv, nq, nkv), tokens))
        if r.random() < 0.5:
            q_out = q
        if r.random() < 0.5:
            k_out = k
        sets = [places(*x, T, n, D) for x, n in zip((q, k, q_out, k_out), (nq, nkv, nq, nkv))]
        # an output's own rows lie one dimension within the other
        nested = all(b >= (n_in - 1) * a + D or n_out == 1 for a, b, n_in, n_out in
                     ((min(x[1], x[2]), max(x[1], x[2]), T if x[1] < x[2] else n, n if x[1] < x[2] else T)
                      for x, n in ((q_out, nq), (k_out, nkv))))
        if not nested or any(len(s) != T * n * (D // 8) for s, n in zip(sets[2:], (nq, nkv))):
            continue
        hit = bool(sets[2] & sets[3] or sets[2] & sets[1] or sets[3] & sets[0] or
                   (q_out != q and sets[2] & sets[0]) or (k_out != k and sets[3] & sets[1]))
        rc = rope(L, T, nq, nkv, D, q, k, q_out, k_out)
        what = (T, nq, nkv, q, k, q_out, k_out, L.moe_last_error())
        if hit:
            assert rc == -2 and b"overlap" in L.moe_last_error(), what
            refused += 1
        elif T == 1 or len({x[1] for x in (q, k, q_out, k_out)}) == 1:
            assert rc in (-4, -6), what
            accepted += 1


def test_heads_of_q_k_and_v_in_turn_may_be_turned_in_place(L):
    """One projection's product [T, heads, (q, k, v), D]."""
    D, H = 64, 8
    q, k = (0, H * 3 * D, 3 * D), (D, H * 3 * D, 3 * D)
    for T in (1, 2, 1000):
        assert rope(L, T, H, H, D, q, k, q, k) in (-4, -6)
        assert rope(L, T, H, H, D, q, k, q, (D - 8, H * 3 * D, 3 * D)) == -2
        assert rope(L, T, H, H, D, q, k, q, (D + 8, H * 3 * D, 3 * D)) == -2
    # heads first: [(q, k), heads, T, D]
    q, k = (0, D, 1000 * D), (H * 1000 * D, D, 1000 * D)
    assert rope(L, 1000, H, H, D, q, k, q, k) in (-4, -6)


def test_attention_outputs_between_the_heads_of_q(L):
    D, H, B = 64, 8, 5
    cache = _KV_CACHE.pack(1 << 20, 1 << 21, moe.MOE_DT_BF16, 1, 50, 16, 2, D, 0, 2048, 128, 64, 1.0, 1.0)
    ws = L.moe_attention_decode_workspace_bytes(H, 2, D)

    def attn(q, out, B=B):
        return L.moe_attention_decode(heads(*q), 0, cache, 0, FAKE, 4, 4, FAKE, B, H, 1.0, 0, heads(*out), None, FAKE, ws, None)

    q = (0, H * 2 * D, 2 * D)
    for n in (1, B):
        assert attn(q, (D, H * 2 * D, 2 * D), n) in (-4, -6)
        assert attn(q, (D - 8, H * 2 * D, 2 * D), n) == -2
        assert attn(q, (0, H * 2 * D, 2 * D), n) == -2
