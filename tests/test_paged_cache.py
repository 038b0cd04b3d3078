"""Bookkeeping of the paged cache on the CPU: random runs of open, append, fork, close and compact against a plain
model of every sequence's tokens, with the page copies done by tensor indexing."""
import random

import pytest
import torch

import mixture_experts_gemv_b200 as moe
from mixture_experts_gemv_b200.paged_cache import PagedKvCache


class CpuOps:
    """moe_copy_pages' definition on CPU tensors, with its refusals."""

    def __init__(self):
        self.copied = 0

    def copy_pages(self, cache, src, dst, block_tables=None):
        assert len(src) == len(dst) and len(set(dst)) == len(dst) and not set(src) & set(dst)
        self.copied += len(src)
        for t in (cache.k, cache.v):
            t[:, dst] = t[:, src]
        if block_tables is not None:
            assert len(set(src)) == len(src)
            to = torch.arange(-1, cache.num_pages, dtype=torch.int32)
            to[torch.tensor(src) + 1] = torch.tensor(dst, dtype=torch.int32)
            block_tables.copy_(to[block_tables.long() + 1])


def build(num_pages=24, page_size=4, max_seqs=6, max_tokens=40, layout="HND"):
    return PagedKvCache(2, num_pages, page_size, 1, 16, max_seqs, max_tokens, dtype=torch.float16, layout=layout, device="cpu",
                        ops=CpuOps())


def write(c, slots, values):
    for layer in range(2):
        for t, sign in ((c.cache.k, 1), (c.cache.v, -1)):
            t = t[layer] if c.cache.layout == "NHD" else t[layer].transpose(1, 2)
            t[slots // c.page_size, slots % c.page_size, 0] = (sign * (values + 100 * layer)).half()[:, None]


def read(c, row, layer, kind):
    n = int(c.seq_lens[row])
    at = torch.arange(n)
    t = getattr(c.cache, kind)[layer]
    t = t if c.cache.layout == "NHD" else t.transpose(1, 2)
    return t[c.block_tables[row].long()[at // c.page_size], at % c.page_size, 0, 0]


@pytest.mark.parametrize("seed,layout,page_size", [(0, "HND", 4), (1, "NHD", 4), (2, "HND", 1), (3, "NHD", 7), (4, "HND", 3)])
def test_random_runs_match_a_plain_model(seed, layout, page_size):
    r = random.Random(seed)
    c = build(num_pages=30, page_size=page_size, layout=layout)
    model, stamp, refused, moved = {}, 0, 0, 0
    for _ in range(400):
        act = r.choice(("open", "append", "append", "append", "fork", "close", "compact"))
        if act == "open" and len(model) < 6:
            model[c.open()] = []
        elif act == "append" and model:
            rows = r.sample(sorted(model), r.randint(1, len(model)))
            counts = [r.choice((0, 1, 1, 2, 5)) for _ in rows]
            before = ([list(c.pages_of(x)) for x in model], c.free_pages, c.block_tables.clone(), c.seq_lens.clone())
            try:
                pos, slots = c.append(rows, counts)
            except moe.MoeError:
                refused += 1
                assert before[0] == [list(c.pages_of(x)) for x in model] and before[1] == c.free_pages
                assert torch.equal(before[2], c.block_tables) and torch.equal(before[3], c.seq_lens)
                continue
            assert pos.dtype == torch.int32 and slots.dtype == torch.int64
            assert pos.tolist() == [len(model[x]) + i for x, n in zip(rows, counts) for i in range(n)]
            assert len(set(slots.tolist())) == sum(counts)
            new = [stamp + i for i in range(sum(counts))]
            stamp = (stamp + sum(counts)) % 1000
            write(c, slots, torch.tensor(new, dtype=torch.float32))
            for x, n in zip(rows, counts):
                model[x] = model[x] + new[:n]
                new = new[n:]
        elif act == "fork" and model and len(model) < 6:
            x = r.choice(sorted(model))
            model[c.fork(x)] = list(model[x])
        elif act == "close" and model and r.random() < 0.5:
            x = r.choice(sorted(model))
            c.close(x)
            del model[x]
        elif act == "compact":
            moved += c.compact()
            used = {p for x in model for p in c.pages_of(x)}
            assert used == set(range(len(used)))
        used = {p for x in model for p in c.pages_of(x)}
        assert len(used) + c.free_pages == c.num_pages
        for x, want in model.items():
            assert c.length(x) == len(want) == int(c.seq_lens[x])
            for layer in range(2):
                assert read(c, x, layer, "k").tolist() == [v + 100 * layer for v in want]
                assert read(c, x, layer, "v").tolist() == [-v - 100 * layer for v in want]
    # all three kinds of trouble were met (a page of one token is never written by two)
    assert refused and moved and (c.ops.copied > moved or page_size == 1)


def test_a_fork_copies_its_last_page_once_and_only_when_written():
    c = build()
    a = c.open()
    c.append([a], [6])           # pages 0 and 1, the second half full
    b = c.fork(a)
    assert c.pages_of(b) == c.pages_of(a) and c.ops.copied == 0
    c.append([a, b], [1, 1])     # the first writer takes a copy, the second one has the page alone then
    assert c.ops.copied == 1 and c.pages_of(a)[0] == c.pages_of(b)[0] and c.pages_of(a)[1] != c.pages_of(b)[1]
    d = c.fork(a)
    c.append([d], [0])
    assert c.ops.copied == 1
    c.close(a)
    c.append([d], [1])           # the other holder has gone
    assert c.ops.copied == 1
    e = c.open()
    c.append([e], [8])           # full pages: a fork's next token goes into a page of its own
    f = c.fork(e)
    c.append([f], [1])
    assert c.ops.copied == 1 and c.pages_of(f)[:2] == c.pages_of(e)


def test_refusals():
    c = build(num_pages=3, max_seqs=2, max_tokens=10)
    with pytest.raises(moe.MoeError):
        c.append([0], [1])       # not open
    a, b = c.open(), c.open()
    for call in (lambda: c.open(), lambda: c.fork(a), lambda: c.append([a], [1, 2]), lambda: c.append([a, a], [1, 1]),
                 lambda: c.append([a], [-1]), lambda: c.append([a], [11]), lambda: c.append([a, b], [9, 4]), lambda: c.close(7)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_BAD_ARG
    assert c.free_pages == 3
    c.append([a, b], [8, 4])
    assert c.free_pages == 0
    with pytest.raises(moe.MoeError):
        PagedKvCache(1, 0, 4, 1, 16, 1, 4, device="cpu", ops=CpuOps())
    with pytest.raises(moe.MoeError):
        PagedKvCache(1, 2, 4, 1, 16, 1, 4, dtype=torch.float32, device="cpu", ops=CpuOps())
