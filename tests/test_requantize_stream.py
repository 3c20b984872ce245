"""requantize_kv_pool_fp4 on a stream of the caller's: nothing is read before it is written,
no memory is used again before it has been read.

The order is shown on the host, with streams and calls that only keep a record; the GPU
test then runs it behind a current stream that is busy."""
import contextlib
import os

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.mark.parametrize("handle", [False, True])
def test_work_is_ordered_between_the_two_streams(L, monkeypatch, handle):
    log = []

    class Stream:
        def __init__(self, name, cuda_stream=0):
            self.name, self.cuda_stream = name, cuda_stream

        def wait_stream(self, other):
            log.append(("wait", self.name, other.name))

    current = [Stream("caller")]

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    def note(what):
        log.append((what, current[-1].name))

    arange, empty = torch.arange, torch.empty
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: Stream("side", h))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", use)
    pool = L.dsv4sa_pool_desc_init(L.POOL_KV, 1 << 20, 1500)
    buf = torch.empty(L.dsv4sa_pool_bytes(L.POOL_KV_FP4, 1500) + 1024, dtype=torch.uint8)
    monkeypatch.setattr(L, "_alloc_pool", lambda *a: buf[-buf.data_ptr() % 1024:])
    monkeypatch.setattr(torch, "arange", lambda *a, **k: (note("fill"), arange(*a, **k))[1])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (note("allocate"), empty(*a, **k))[1])
    for name in ("dsv4sa_cache_read", "dsv4sa_cache_write"):
        monkeypatch.setattr(L, name, lambda *a, name=name: note(name))   # no stream named: the current one

    L.requantize_kv_pool_fp4(pool, "cpu", 77 if handle else Stream("side"))
    assert log[0] == ("wait", "side", "caller") and log[-1] == ("wait", "caller", "side")
    assert {e[-1] for e in log[1:-1]} == {"side"}, log
    calls = [e[0] for e in log if e[0].startswith("dsv4sa")]
    assert calls == ["dsv4sa_cache_read", "dsv4sa_cache_write"] * 2      # 1500 pages, 1024 at a time

    log.clear()
    L.requantize_kv_pool_fp4(pool, "cpu")                                # none given: no order to make
    assert {e[-1] for e in log} == {"caller"} and not [e for e in log if e[0] == "wait"]


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_side_stream_behind_a_busy_current_one(L, handle):
    rng = np.random.default_rng(3)
    P = 2100                                                             # three passes, the last a short one
    codes = rng.integers(0, 0x7F, (P, 64, 448)).astype(np.uint8)
    scale = rng.uniform(0.01, 2, (P, 64, 7)).astype(np.float32)
    rope = rng.integers(0, 0x7F00, (P, 64, 64)).astype(np.uint16)
    buf, d = L.pack_kv_pool(codes, scale, rope)
    want, _ = L.requantize_kv_pool_fp4(d)
    later = L._alloc_pool(L.POOL_KV, P, "cuda")
    d2 = L.dsv4sa_pool_desc_init(L.POOL_KV, later, P)
    later.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                                        # some ten milliseconds
    later.copy_(buf)                                                     # the pool is only then written
    got, _ = L.requantize_kv_pool_fp4(d2, stream=side.cuda_stream if handle else side)
    other = torch.full((P * 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")   # may take the memory given back
    page = L._layout(L.POOL_KV_FP4, P).page_stride
    both = torch.stack((got, want)).view(2, P, page)                     # on the current stream, which has waited
    torch.cuda.synchronize()
    pad = torch.ones(page, dtype=torch.bool)
    pad[22528:].view(64, 16)[:, 14:] = False                             # the padding of the scale rows is never written
    assert torch.equal(both[0][:, pad.cuda()], both[1][:, pad.cuda()])
    assert float(other.min()) == 7.0 and L.dsv4sa_check_errors() == (0, 0)
