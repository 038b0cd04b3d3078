"""Measured cases of the attention operators beside the routed layer: per-head norm and rotation with the append to
a paged cache, attention of one new token over that cache, and copies and moves of its pages.

`run` computes a case in plain torch operations (`own` false) or through this package's entry points (`own` true).
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
EPS = 1e-6
SCALES = {"bf16": (1.0, 1.0), "fp16": (1.0, 1.0), "e4m3": (0.0625, 0.03125)}


# ------------------------------------------------------------------ cases

def _attn(B, longest, nq, nkv, D, q, cache, page, layout="NHD", window=0, shortest=1):
    return {"op": "attention", "B": B, "longest": longest, "shortest": shortest, "nq": nq, "nkv": nkv, "D": D, "q": q,
            "cache": cache, "page": page, "layout": layout, "window": window}


def _rope(T, nq, nkv, D, rot, interleaved, x, cache, page, layout="NHD", far=0, base=10000.0, factor=1.0, norm=True):
    return {"op": "rope", "T": T, "nq": nq, "nkv": nkv, "D": D, "rot": rot, "interleaved": interleaved, "x": x,
            "cache": cache, "page": page, "layout": layout, "far": far, "base": base, "factor": factor, "norm": norm}


def _pages(layers, pages, n, nkv, D, cache, page, B, move, layout="NHD"):
    return {"op": "pages", "layers": layers, "pages": pages, "n": n, "nkv": nkv, "D": D, "cache": cache, "page": page,
            "B": B, "move": move, "layout": layout}


def listed():
    return [
        # one chat request early in its answer: latency
        dict(_attn(1, 997, 16, 8, 128, "bf16", "bf16", 16, shortest=997), name="attn_one_997"),
        # one request behind the 10,000-token prompt
        dict(_attn(1, 10000, 16, 8, 256, "bf16", "bf16", 16, "HND", shortest=10000), name="attn_one_10000"),
        # one request behind the 40,000-token prompt, wide heads shared by eight queries each
        dict(_attn(1, 40000, 16, 2, 512, "bf16", "bf16", 16, shortest=40000), name="attn_one_40000_wide"),
        # eight concurrent requests of very different ages, one of them not begun
        dict(_attn(8, 40000, 32, 8, 128, "fp16", "fp16", 16, shortest=0), name="attn_8_ragged"),
        # sliding-window layer, 32 requests, large pages
        dict(_attn(32, 10000, 16, 8, 256, "bf16", "bf16", 64, "HND", window=1024, shortest=100), name="attn_32_window"),
        # a full batch over an 8-bit cache
        dict(_attn(128, 4096, 32, 4, 128, "bf16", "e4m3", 32, shortest=500), name="attn_128_e4m3"),
        # eight tokens of a decode step
        dict(_rope(8, 16, 8, 256, 256, False, "bf16", "bf16", 16, far=9000), name="rope_8"),
        # a 4,096-token prompt
        dict(_rope(4096, 32, 8, 128, 128, False, "bf16", "bf16", 16), name="rope_4096"),
        # a 10,000-token prompt chunk far into a long context: part of the head, pairs interleaved, frequencies
        # interpolated, 8-bit cache
        dict(_rope(10000, 16, 2, 512, 128, True, "fp16", "e4m3", 64, "HND", far=240000, base=1000000.0, factor=8.0),
             name="rope_10000_partial"),
        # eight requests fork: their last pages are copied in all 30 layers
        dict(_pages(30, 64, 8, 8, 256, "bf16", 16, 8, False), name="pages_fork_8"),
        # compaction: live pages move down into holes and the tables follow, five layers
        dict(_pages(5, 2048, 601, 8, 256, "bf16", 16, 32, True, "HND"), name="pages_compact_601"),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "rope", "pages"))
    layout = rng.choice(("NHD", "HND"))
    page = rng.choice((8, 16, 24, 32, 64, 128))
    D = rng.choice((64, 96, 128, 256, 512))
    if op == "attention":
        x = rng.choice(("bf16", "fp16"))
        nkv = rng.choice((1, 2, 4, 8))
        nq = nkv * rng.choice((1, 2, 4, 6, 8, 16))
        B = _log_between(rng, 1, 128)
        # the K and V of the longest possible batch stay under those of the largest listed case
        most = max(64, min(40000, int(2.3e8 / (B * nkv * D * 4))))
        longest = _log_between(rng, 32, most)
        return _attn(B, longest, nq, nkv, D, x, rng.choice((x, x, "e4m3")), page, layout,
                     rng.choice((0, 0, 1024, 127)), min(longest, rng.choice((0, 1, longest // 2))))
    if op == "rope":
        x = rng.choice(("bf16", "fp16"))
        nkv = rng.choice((1, 2, 4, 8))
        nq = nkv * rng.choice((1, 2, 4, 8))
        most = max(2, min(10000, int(1.0e8 / ((nq + 2 * nkv) * D))))
        return _rope(_log_between(rng, 1, most), nq, nkv, D, rng.choice((D, D, D // 2, 32)), rng.random() < 0.5, x,
                     rng.choice((x, x, "e4m3")), page, layout, rng.choice((0, 1000, 200000)),
                     rng.choice((10000.0, 500000.0)), rng.choice((1.0, 4.0)), rng.random() < 0.8)
    nkv = rng.choice((1, 2, 8))
    cache = rng.choice(("bf16", "fp16", "e4m3"))
    layers = _log_between(rng, 1, 30)
    most = max(4, min(600, int(4.0e8 / (layers * page * nkv * D * BYTES[cache] * 4))))
    n = _log_between(rng, 1, most)
    return _pages(layers, 3 * n + rng.randrange(1, 9), n, nkv, D, cache, page, _log_between(rng, 1, 64),
                  rng.random() < 0.5, layout)


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The case's lengths: spread evenly over their logarithm, the longest and the shortest among them."""
    B, lo, hi = c["B"], c["shortest"], c["longest"]
    r = random.Random(B * 1000003 + hi)
    if B == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    got = [int(math.exp(a + (b - a) * i / (B - 1) + 1e-9)) - 1 for i in range(B)]
    got[0], got[-1] = lo, hi
    r.shuffle(got)
    return got


def _normal(g, shape, dtype, dev):
    """Normal values of the type; 8-bit ones spread over the codes that a scaled cache uses."""
    if dtype == torch.float8_e4m3fn:
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) * 16).clamp(-448, 448).to(dtype)
    return torch.randn(shape, generator=g, device=dev, dtype=dtype)


def _cache_shape(c, pages):
    return (pages, c["page"], c["nkv"], c["D"]) if c["layout"] == "NHD" else (pages, c["nkv"], c["page"], c["D"])


def _inv_freq(c, dev):
    """Frequencies of the rotation; beyond factor 1 interpolated linearly."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
    return c["base"] ** (-2.0 * i / c["rot"]) / c["factor"]


def prepare(case, seed):
    c, dev = case, "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    host = random.Random(int(seed))
    s = {"case": c, "device": dev}
    ks, vs = SCALES[c["cache"]]
    s["k_scale"], s["v_scale"] = ks, vs
    dt = DTYPES[c["cache"]]
    if c["op"] == "attention":
        lens = _lengths(c)
        need = [-(-n // c["page"]) for n in lens]
        cols = max(1, max(need))
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        used = torch.arange(cols, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
        tables = torch.full((c["B"], cols), -1, dtype=torch.int32, device=dev)
        tables[used] = order[: sum(need)]
        s["tables"] = tables
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = (torch.randn((c["B"], c["nq"], c["D"]), generator=g, device=dev) * 2.5).to(DTYPES[c["q"]])
        s["scale"] = c["D"] ** -0.5
        s["k"], s["v"] = (_normal(g, _cache_shape(c, pages), dt, dev) for _ in range(2))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["B"], c["nq"]), dtype=torch.float32, device=dev)
    elif c["op"] == "rope":
        T, x = c["T"], DTYPES[c["x"]]
        # q, k and v are parts of the rows of one projection's product
        qkv = torch.randn((T, c["nq"] + 2 * c["nkv"], c["D"]), generator=g, device=dev).to(x)
        s["q"], s["k_new"], s["v_new"] = qkv.split((c["nq"], c["nkv"], c["nkv"]), dim=1)
        pages = -(-T // c["page"]) + 3
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        slots = order[t // c["page"]] * c["page"] + t % c["page"]
        if T > 2:
            slots[host.randrange(T)] = -1  # a padded row
        s["slots"] = slots
        s["positions"] = (t + c["far"] + host.randrange(100)).to(torch.int32)
        s["inv_freq"] = _inv_freq(c, dev)
        s["q_gain"], s["k_gain"] = (1 + 0.2 * torch.randn(c["D"], generator=g, device=dev) if c["norm"] else None
                                    for _ in range(2))
        s["k"], s["v"] = (_normal(g, _cache_shape(c, pages), dt, dev) for _ in range(2))
        s["out"] = torch.empty((T, c["nq"], c["D"]), dtype=x, device=dev)
    else:
        shape = (c["layers"],) + _cache_shape(c, c["pages"])
        s["k"], s["v"] = (_normal(g, shape, dt, dev) for _ in range(2))
        order = list(range(c["pages"]))
        host.shuffle(order)
        # the lists of pages are the scheduler's: they are on the host
        s["src"], s["dst"] = (torch.tensor(order[i: i + c["n"]], dtype=torch.int32) for i in (0, c["n"]))
        live = torch.tensor(order[: c["n"]] + order[2 * c["n"]:], dtype=torch.int32, device=dev)
        at = torch.randint(len(live), (c["B"], max(1, c["pages"] // c["B"])), generator=g, device=dev)
        s["tables"] = live[at].contiguous() if c["move"] else None
    return s


# ------------------------------------------------------------------ the plain forms

def _gathered(cache, tables, c):
    """The rows of the sequences' pages in order, [B, L, nkv, D] in 32 bits."""
    got = cache.view(torch.uint8)[tables.clamp(min=0).long()].view(cache.dtype)
    if c["layout"] == "HND":
        got = got.transpose(2, 3)
    return got.reshape(got.shape[0], -1, c["nkv"], c["D"]).float()


def _plain_attention(s):
    c = s["case"]
    k, v = _gathered(s["k"], s["tables"], c) * s["k_scale"], _gathered(s["v"], s["tables"], c) * s["v_scale"]
    B, L = k.shape[:2]
    at = torch.arange(L, device=k.device)[None, :]
    lens = s["lens"][:, None]
    seen = at < lens
    if c["window"]:
        seen = seen & (at >= lens - c["window"])
    v = v * seen[:, :, None, None]
    q = s["q"].float().view(B, c["nkv"], -1, c["D"])
    score = torch.einsum("bhgd,blhd->bhgl", q, k) * s["scale"]
    score = score.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.log(total) + top
    return out.reshape(B, -1, c["D"]).to(s["q"].dtype), lse.reshape(B, -1)


def _plain_rotated(x, gain, s):
    c = s["case"]
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
    turn = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(turn).float()[:, None, :], torch.sin(turn).float()[:, None, :]
    rot, rest = x[..., : c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = rot.chunk(2, -1)
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, rest), -1)


def _stored(x, cache, scale):
    """Values as the cache holds them: rounded once, 8-bit ones scaled and saturated first."""
    if cache.dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-448, 448).to(cache.dtype)
    return x.to(cache.dtype)


def _plain_put(cache, rows, s):
    c = s["case"]
    ok = s["slots"] >= 0
    at, rows = s["slots"][ok], rows[ok].view(torch.uint8)
    flat = cache.view(torch.uint8)
    if c["layout"] == "NHD":
        flat[at // c["page"], at % c["page"]] = rows
    else:
        flat[at // c["page"], :, at % c["page"]] = rows


def _plain_rope(s):
    q = _plain_rotated(s["q"], s["q_gain"], s).to(s["q"].dtype)
    k = _plain_rotated(s["k_new"], s["k_gain"], s)
    _plain_put(s["k"], _stored(k, s["k"], s["k_scale"]), s)
    _plain_put(s["v"], _stored(s["v_new"].float(), s["v"], s["v_scale"]), s)
    return q, s["k"], s["v"]


def _plain_pages(s):
    src, dst = (s[n].to(s["device"]).long() for n in ("src", "dst"))
    for cache in (s["k"].view(torch.uint8), s["v"].view(torch.uint8)):
        cache[:, dst] = cache[:, src]
    if s["tables"] is None:
        return s["k"], s["v"]
    to = torch.arange(s["case"]["pages"], dtype=torch.int32, device=s["device"])
    to[src] = dst.to(torch.int32)
    s["tables"] = to[s["tables"].long()]
    return s["k"], s["v"], s["tables"]


# ------------------------------------------------------------------ a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attention": _plain_attention, "rope": _plain_rope, "pages": _plain_pages}[c["op"]](s)
    import mixture_experts_gemv_b200 as moe
    if c["op"] == "attention":
        cache = moe.MoeKvCache(s["k"], s["v"], c["layout"], s["k_scale"], s["v_scale"])
        moe.moe_attention_decode(s["q"], cache, s["tables"], s["lens"], s["out"], scale=s["scale"],
                                 window=c["window"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "rope":
        cache = moe.MoeKvCache(s["k"], s["v"], c["layout"], s["k_scale"], s["v_scale"])
        moe.moe_qk_norm_rope(s["q"], s["k_new"], s["v_new"], s["positions"], s["inv_freq"], q_gain=s["q_gain"],
                             k_gain=s["k_gain"], eps=EPS, interleaved=c["interleaved"], q_out=s["out"], cache=cache,
                             slots=s["slots"])
        return s["out"], s["k"], s["v"]
    cache = moe.MoeKvCache(s["k"], s["v"], c["layout"], s["k_scale"], s["v_scale"])  # all layers
    moe.moe_copy_pages(cache, s["src"], s["dst"], block_tables=s["tables"])
    return (s["k"], s["v"]) if s["tables"] is None else (s["k"], s["v"], s["tables"])


def work(case):
    c = case
    if c["op"] == "attention":
        lens = [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]
        rows = sum(lens)
        table = 4 * sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 2 * rows * c["nkv"] * c["D"] * BYTES[c["cache"]] + table + 4 * c["B"]
                + c["B"] * c["nq"] * (4 * c["D"] + 4), "flops": 4 * rows * c["nq"] * c["D"]}
    if c["op"] == "rope":
        T, D = c["T"], c["D"]
        return {"bytes": T * D * (4 * c["nq"] + 2 * c["nkv"] * (2 + BYTES[c["cache"]])) + T * 12
                + 8 * c["D"] + 4 * c["rot"], "flops": T * D * 8 * (c["nq"] + c["nkv"])}
    page = c["layers"] * c["page"] * c["nkv"] * c["D"] * BYTES[c["cache"]] * 2
    table = 8 * c["B"] * max(1, c["pages"] // c["B"]) if c["move"] else 0
    return {"bytes": 2 * c["n"] * page + table, "flops": 0}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "attention":
        return _exact_attention(s, c)
    if c["op"] == "rope":
        return _exact_rope(s, c)
    for cache in (s["k"], s["v"]):
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            cache[:, b].view(torch.uint8).copy_(cache[:, a].view(torch.uint8))
    if s["tables"] is None:
        return s["k"], s["v"]
    moved = dict(zip(s["src"].tolist(), s["dst"].tolist()))
    rows = [[moved.get(e, e) for e in row] for row in s["tables"].tolist()]
    return s["k"], s["v"], torch.tensor(rows, dtype=torch.int32)


def _exact_attention(s, c):
    outs, lses = [], []
    heads_first = c["layout"] == "HND"
    group = c["nq"] // c["nkv"]
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            outs.append(torch.zeros(c["nq"], c["D"], dtype=torch.float64, device=s["device"]))
            lses.append(torch.full((c["nq"],), float("-inf"), dtype=torch.float64, device=s["device"]))
            continue
        at = torch.arange(first, n, device=s["device"])
        page, off = s["tables"][b].long()[at // c["page"]], at % c["page"]
        rows = []
        for cache, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            raw = cache.view(torch.uint8)
            got = raw[page, :, off] if heads_first else raw[page, off]
            rows.append(got.view(cache.dtype).double().permute(1, 0, 2) * scale)  # [nkv, n, D]
        k, v = rows
        score = (s["q"][b].double().view(c["nkv"], group, c["D"]) @ k.transpose(1, 2)) * s["scale"]
        lse = torch.logsumexp(score, -1)
        outs.append((torch.exp(score - lse[..., None]) @ v).reshape(c["nq"], c["D"]))
        lses.append(lse.reshape(-1))
    return torch.stack(outs), torch.stack(lses)


def _exact_rope(s, c):
    half = c["rot"] // 2
    first = torch.arange(half, device=s["device"])
    first, second = (2 * first, 2 * first + 1) if c["interleaved"] else (first, first + half)
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]

    def rotate(x, gain):
        x = x.double()
        if gain is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS) * gain.double()
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def kept(cache, rows, scale):
        full = cache.double() if cache.dtype != torch.float8_e4m3fn else cache.float().double()
        if cache.dtype == torch.float8_e4m3fn:
            rows = (rows / scale).clamp(-448, 448).float().to(cache.dtype).float().double()
        seq = full if c["layout"] == "NHD" else full.transpose(1, 2)  # [pages, page, nkv, D]
        good = s["slots"] >= 0
        at = s["slots"][good]
        seq[at // c["page"], at % c["page"]] = rows[good]
        return seq if c["layout"] == "NHD" else seq.transpose(1, 2)

    return (rotate(s["q"], s["q_gain"]), kept(s["k"], rotate(s["k_new"], s["k_gain"]), s["k_scale"]),
            kept(s["v"], s["v_new"].double(), s["v_scale"]))
