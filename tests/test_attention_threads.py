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
    torch.cuda.synchronize()
    moe.moe_profile_end()
    moe.moe_destroy()
    assert n == 4 * 500
