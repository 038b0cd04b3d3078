"""Plain 64-bit forms of the attention operators, with the error bounds that their kernels' roundings allow.

A rounding to type t is off by at most eps(t) / 2 of the value (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""
from __future__ import annotations

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
U32 = 2.0 ** -24


def values(t):
    """A tensor's values in 64 bits (8-bit ones through 32)."""
    return t.float().double() if t.dtype == torch.float8_e4m3fn else t.double()


def cache_rows(cache, layer, kind, page, off):
    """Rows (page[i], off[i]) of one layer's K or V as [n, n_kv, D] values times the scale."""
    t = getattr(cache, kind)
    t = t if t.dim() == 4 else t[layer]
    raw = t.view(torch.uint8)
    got = raw[page, off] if cache.layout == "NHD" else raw[page, :, off]
    scale = cache.k_scale if kind == "k" else cache.v_scale
    return values(got.contiguous().view(t.dtype)) * scale


def attention(q, cache, tables, lens, scale, window=0, layer=0):
    """(out, lse, bound on out, bound on lse), 64 bits.

    Bound: every probability is rounded once to the 16-bit type of the V product (u_p), the output once (u_o);
    in 32 bits a score is a sum of D products (D + 8 roundings of sums of |q k|, taken twice over for the
    tensor cores' truncating adds), scaled and shifted (4 roundings of its size), and sums over the n keys
    add at most n / 16 + 64 roundings, likewise twice over; exp2 is good to 2^-22."""
    B, nq, D = q.shape
    group = nq // cache.n_kv
    u_o = HALF_STEP[q.dtype]
    u_p = HALF_STEP[torch.float16] if cache.dtype == torch.float8_e4m3fn else HALF_STEP[cache.dtype]
    out = torch.zeros(B, nq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, nq), float("-inf"), dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    for b, n in enumerate(lens.tolist()):
        lo = max(0, n - window) if window else 0
        if n <= 0:
            continue
        at = torch.arange(lo, n, device=q.device)
        page, off = tables[b].long()[at // cache.page_size], at % cache.page_size
        k = cache_rows(cache, layer, "k", page, off).transpose(0, 1)   # [nkv, n, D]
        v = cache_rows(cache, layer, "v", page, off).transpose(0, 1)
        qb = q[b].double().view(cache.n_kv, group, D)
        s = scale * (qb @ k.transpose(1, 2))
        size = abs(scale) * (qb.abs() @ k.abs().transpose(1, 2))
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[..., None])
        d_s = (2 * (D + 8) * size + 4 * s.abs()).amax(-1) * U32   # [nkv, group]
        rest = 2 * d_s + 2 * (at.numel() / 16 + 64) * U32 + 2.0 ** -21
        a = p @ v.abs()
        o = p @ v
        out[b] = o.reshape(nq, D)
        tol[b] = (a * (u_p + rest[..., None]) + u_o * o.abs() + 1e-30).reshape(nq, D) * 1.01
        lse[b] = l.reshape(nq)
        lse_tol[b] = (rest + 4 * U32 * l.abs()).reshape(nq)
    return out, lse, tol, lse_tol


def rotated(x, gain, eps, positions, inv_freq, interleaved, rope_scale=1.0):
    """(y, size): norm and rotation in 64 bits, and |terms| of each output for bounds in 32 bits."""
    u = x.double()
    if gain is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * gain.double()
    size = u.abs()
    if inv_freq is None:
        return u, size
    half = inv_freq.numel()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    turn = (positions.double()[:, None] * inv_freq[None])[:, None, :]
    c, s = torch.cos(turn) * rope_scale, torch.sin(turn) * rope_scale
    y, size = u.clone(), size.clone()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    both = (u[..., a].abs() + u[..., b].abs()) * abs(rope_scale)
    size[..., a] = both
    size[..., b] = both
    return y, size


def rotated_bound(y, size, D, dtype, scale=1.0):
    """Norm: D + 8 roundings in the sum of squares (half of them on the root), 8 more for root, quotient, gain
    and rotation, sine and cosine good to 2^-22 of the values turned; one rounding to the type (e4m3: of
    value / scale, with half a step of its subnormals, 2^-10)."""
    tol32 = size * ((D / 2 + 16) * U32 + 2.0 ** -21)
    if dtype == torch.float8_e4m3fn:
        return tol32 + y.abs() * 2.0 ** -4 + scale * 2.0 ** -10 + 1e-30
    # a bf16 or fp16 result below the smallest normal number is off by half a step of the subnormals
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-40
    return (tol32 + (y.abs() + tol32) * HALF_STEP[dtype] + tiny) * 1.01


def stored(y, dtype, scale):
    """What a cache of that type keeps of values y, as values."""
    if dtype == torch.float8_e4m3fn:
        return (y / scale).clamp(-448, 448)
    return y
