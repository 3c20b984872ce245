"""The device error words of all kernel files, read and cleared by one call."""
import threading
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bad_position(L):
    cs = torch.zeros(2, 8, 2, device="cuda")
    L.dsv4sa_rope(torch.zeros(1, 1, 16, dtype=torch.bfloat16, device="cuda"), cs, i32(5))


def bad_bounds(L):
    idx = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    L.dsv4sa_tree_window_indices(i32(0, 9), i32(0), i32(0), 2, 0, 0, 2, idx)


def bad_row(L):
    buf = L._alloc_pool(L.POOL_KV, 1, "cuda")
    pool = L.dsv4sa_pool_desc_init(L.POOL_KV, buf, 1)
    L.dsv4sa_cache_append(pool, i32(0).view(1, 1), i32(0), i32(64), torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda"))


def test_any_file_is_heard_and_cleared(L):
    assert L.dsv4sa_check_errors() == (0, 0)
    for calls in ((bad_position,), (bad_bounds,), (bad_row,), (bad_position, bad_bounds, bad_row)):
        for f in calls:
            f(L)
        assert L.dsv4sa_check_errors() == (5, 1)
        assert L.dsv4sa_check_errors() == (0, 0)
    res = i32(7)
    L.dsv4sa_selftest_wait_timeout(res)              # two bits of two files
    bad_row(L)
    assert L.dsv4sa_check_errors() == (6, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bad_position(L)
    assert L.dsv4sa_check_errors(s) == (5, 1)
    assert L.dsv4sa_check_errors() == (0, 0)


def test_threads_that_check_at_once(L):
    """Each error is seen by one of them, and by one only."""
    seen, rounds = [], 60
    gate = threading.Barrier(9)

    def work():
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        mine = []
        for _ in range(rounds):
            gate.wait(60)
            mine.append(L.dsv4sa_check_errors(s))
            gate.wait(60)
        seen.append(mine)
    threads = [threading.Thread(target=work) for _ in range(8)]
    for t in threads:
        t.start()
    for r in range(rounds):
        if r % 3:
            bad_position(L)
            torch.cuda.synchronize()
        gate.wait(60)
        gate.wait(60)
    for t in threads:
        t.join()
    assert len(seen) == 8
    for r in range(rounds):
        got = [m[r] for m in seen]
        assert sorted(got) == [(0, 0)] * (7 if r % 3 else 8) + ([(5, 1)] if r % 3 else []), (r, got)


def test_a_check_costs_a_few_small_copies(L):
    """Not one copy and one wait for each kernel file (eleven): the call stands in a server's step."""
    word, host = i32(0), torch.zeros(1, dtype=torch.int32)

    def copy():
        host.copy_(word)

    def median(f):
        for _ in range(30):
            f()
        ts = []
        for _ in range(40):
            t = time.perf_counter()
            for _ in range(10):
                f()
            ts.append(time.perf_counter() - t)
        return float(np.median(ts))
    torch.cuda.synchronize()
    assert median(L.dsv4sa_check_errors) <= 5 * median(copy)
