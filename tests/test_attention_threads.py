"""The attention entry points called from several host threads: each reads its own error text, and no launch goes uncounted."""
import ctypes
import threading

import pytest
import torch

import mixture_experts_gemv_b200 as moe


@pytest.fixture(scope="module")
def L():
    from mixture_experts_gemv_b200 import build
    build.build()
    return moe.lib()


def in_thread(fn):
    got = []
    t = threading.Thread(target=lambda: got.append(fn()))
    t.start()
    t.join()
    return got[0]


def test_a_threads_error_text_is_its_own(L):
    f, s = (ctypes.c_double * 1)(), ctypes.c_float()

    def refused(kind):
        assert L.moe_rope_frequencies(kind, 2, 10.0, 1.0, 1.0, 2.0, 1.0, f, ctypes.byref(s)) == moe.MOE_ERR_BAD_ARG
        return L.moe_last_error().decode()

    first = refused(7)
    assert "7" in first
    other = in_thread(lambda: refused(9))
    assert "9" in other and other != first
    assert L.moe_last_error().decode() == first
    assert in_thread(lambda: L.moe_last_error().decode()) == ""   # a thread without a failure


@pytest.mark.parametrize("threads", [8])
def test_threads_that_are_refused_at_once(L, threads):
    f, s = (ctypes.c_double * 1)(), ctypes.c_float()
    start = threading.Barrier(threads)
    wrong = []

    def run(i):
        start.wait()
        for n in range(500):
            kind = 1000 * (i + 1) + n % 7
            L.moe_rope_frequencies(kind, 2, 10.0, 1.0, 1.0, 2.0, 1.0, f, ctypes.byref(s))
            text = L.moe_last_error().decode(errors="replace")
            if not text.endswith(f" {kind}"):
                wrong.append((kind, text))

    all_ = [threading.Thread(target=run, args=(i,)) for i in range(threads)]
    for t in all_:
        t.start()
    for t in all_:
        t.join()
    assert not wrong, wrong[:5]


@pytest.mark.gpu
def test_launches_of_several_threads_are_all_counted(L):
    moe.moe_init(0, 1, 32, 32, 1, 1)
    caches = []
    for _ in range(4):
        k = torch.zeros(4, 1, 1, 16, device="cuda:0", dtype=torch.bfloat16)
        caches.append((moe.MoeKvCache(k, k.clone()), torch.cuda.Stream()))
    torch.cuda.synchronize()
    moe.moe_profile_begin()

    def run(cache, stream):
        for _ in range(500):
            moe.moe_copy_pages(cache, [0], [1], stream=stream)

    all_ = [threading.Thread(target=run, args=c) for c in caches]
    for t in all_:
        t.start()
    for t in all_:
        t.join()
    n = moe.moe_profile_kernel_launches()
    moe.moe_cache_check()   # one kernel too
    with_check = moe.moe_profile_kernel_launches()
    moe.moe_profile_end()
    moe.moe_destroy()
    assert n == 4 * 500 and with_check == n + 1


@pytest.mark.gpu
def test_no_error_is_lost_between_checks_of_two_threads(L):
    """A check takes the error word and clears it at once: while another thread checks all the time, each error that is
    raised here is reported, there or here."""
    k = torch.zeros(4, 16, 1, 64, device="cuda:0", dtype=torch.bfloat16)
    cache = moe.MoeKvCache(k, k.clone())
    new = torch.zeros(1, 1, 64, device="cuda:0", dtype=torch.bfloat16)
    out = torch.zeros_like(new)
    past = torch.tensor([64], device="cuda:0")                               # a slot past the cache
    table = torch.tensor([[9]], device="cuda:0", dtype=torch.int32)          # a page that is not there
    one = torch.tensor([1], device="cuda:0", dtype=torch.int32)
    ws = torch.empty(moe.moe_attention_decode_workspace_bytes(1, 1, 64), device="cuda:0", dtype=torch.uint8)
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    moe.moe_cache_check()
    seen, stop = {"slot": 0, "block-table": 0}, threading.Event()
    lock = threading.Lock()

    def check(stream):
        try:
            moe.moe_cache_check(stream=stream)
        except moe.MoeError as e:
            with lock:
                for kind in seen:
                    seen[kind] += kind in str(e)

    def keep_checking():
        while not stop.is_set():
            check(other)

    def keep_busy():   # the other stream always has about 0.2 ms of work queued, whatever the check enqueues next
        events = []
        with torch.cuda.stream(other):
            while not stop.is_set():
                torch.cuda._sleep(100000)
                events.append(torch.cuda.Event())
                events[-1].record()
                if len(events) > 4:
                    events.pop(0).synchronize()

    threads = [threading.Thread(target=f) for f in (keep_busy, keep_checking)]
    for t in threads:
        t.start()
    lost = 0
    try:
        for i in range(400):
            kind = ("slot", "block-table")[i % 2]
            with lock:
                before = seen[kind]
            if i % 2 == 0:
                moe.moe_qk_norm_rope(None, new, new, None, None, cache=cache, slots=past, stream=mine)
            else:
                moe.moe_attention_decode(new, cache, table, one, out, 1.0, workspace=ws, stream=mine)
            mine.synchronize()
            check(mine)
            for _ in range(200):   # the other thread may have taken it, and be on its way to count it
                if seen[kind] != before:
                    break
                stop.wait(0.001)
            lost += seen[kind] == before
    finally:
        stop.set()
        for t in threads:
            t.join()
    assert lost == 0
    moe.moe_cache_check()


@pytest.mark.gpu
def test_a_check_under_capture_is_refused_and_leaves_the_capture_whole(L):
    k = torch.ones(4, 16, 1, 64, device="cuda:0", dtype=torch.bfloat16)
    k[1] = 2
    cache = moe.MoeKvCache(k, k.clone())
    moe.moe_copy_pages(cache, [0], [2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_copy_pages(cache, [1], [3])
        with pytest.raises(moe.MoeError) as e:
            moe.moe_cache_check()
        assert "captured" in str(e.value)
    graph.replay()
    assert (k[3] == 2).all()
    moe.moe_cache_check()
