"""Long appends, where a warp takes a batch of consecutive rows through its ring of stages: the same bytes
as the same rows in calls of a few hundred, where each warp has one (those are held against the
oracle in test_gpu_append.py)."""
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


def case(L, n, kind, seed, bad=True):
    """Lists of n rows into 7 sequences of a random page table; here and there padding, and rows that no slot, page,
    position or source has -- several in a row, too, and the first and the last."""
    rng = np.random.default_rng(seed)
    B, table = 7, 5000
    per = -(-n // B // 64) + 2
    pages = B * per
    pt = rng.permutation(pages).reshape(B, per).astype(np.int32)
    pt[3, 0] = pages                                       # one page that is out of range
    slots = rng.permutation(B * per * 64)[:n]
    seq, ent = (slots // (per * 64)).astype(np.int32), (slots % (per * 64)).astype(np.int32)
    pos = rng.integers(0, table, n).astype(np.int32)
    src = rng.integers(0, n, n).astype(np.int32)
    if bad:
        kinds = rng.integers(0, 60, n)
        kinds[:3], kinds[-2:] = 0, 1
        kinds[100:130] = 0
        kinds[200:233] = 1
        seq[kinds == 0] = -1
        ent[kinds == 1] = per * 64
        ent[kinds == 2] = -3
        pos[kinds == 3] = table
        src[kinds == 4] = n
        seq[kinds == 5] = B
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn(n, 520, generator=g, device="cuda").to(torch.bfloat16)
    cs = torch.empty(table, 32, 2, device="cuda")
    L.dsv4sa_rope_table(cs, base=160000.0, factor=16.0, original_len=65536)
    w = 1 + 0.2 * torch.randn(512, generator=g, device="cuda")
    return dict(pt=up(pt), seq=up(seq), ent=up(ent), pos=up(pos), src=up(src), rows=wide[:, 8:], cs=cs, w=w, pages=pages, kind=kind)


def pool(L, c):
    buf = L._alloc_pool(c["kind"], c["pages"], "cuda")
    buf.fill_(0x5A)
    return buf, L.dsv4sa_pool_desc_init(c["kind"], buf, c["pages"])


def append(L, c, desc, a, b, norm, rotate, select, stream=None):
    rows = c["rows"] if select else c["rows"][a:]
    L.dsv4sa_cache_append(desc, c["pt"], c["seq"][a:b], c["pos"][a:b], rows, c["cs"] if rotate else None, row_entry=c["ent"][a:b],
                          src_row=c["src"][a:b] if select else None, eps=1e-6 if norm else None, norm_w=c["w"] if norm else None, stream=stream)


@pytest.mark.parametrize("norm,rotate,select", [(True, True, False), (True, True, True), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("n", [4799, 4865, 20011, 77777])
def test_batches_of_rows(L, n, kind, norm, rotate, select):
    c = case(L, n, kind, n)
    buf, desc = pool(L, c)
    append(L, c, desc, 0, n, norm, rotate, select)
    assert L.dsv4sa_check_errors() == (5, 1)
    want, wdesc = pool(L, c)
    for a in range(0, n, 701):
        append(L, c, wdesc, a, min(n, a + 701), norm, rotate, select)
    assert L.dsv4sa_check_errors() == (5, 1)
    assert torch.equal(buf, want)
    assert (buf != 0x5A).any()


@pytest.mark.parametrize("kind,norm", [(0, True), (3, True), (0, False), (3, False)])
def test_more_rows_than_run_at_once(L, kind, norm):
    """Above 16 rows a warp, 8 warps a CTA and 16 CTAs a multiprocessor: a warp comes back for another batch."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 16 * 8 * 16 + 5003
    c = case(L, n, kind, 5)
    buf, desc = pool(L, c)
    append(L, c, desc, 0, n, norm, True, False)
    want, wdesc = pool(L, c)
    for a in range(0, n, 4001):
        append(L, c, wdesc, a, min(n, a + 4001), norm, True, False)
    assert L.dsv4sa_check_errors() == (5, 1)
    assert torch.equal(buf, want)


def test_no_error_without_a_bad_row_and_in_a_graph(L):
    n = 30011
    c = case(L, n, 0, 9, bad=False)
    c["pt"][3, 0] = c["pages"] - 1
    keep = c["pt"].flatten() == c["pages"] - 1             # the page that is there twice now: its rows are left out
    twice = keep.view(c["pt"].shape)[c["seq"].long(), (c["ent"] // 64).long()]
    c["seq"][twice] = -1
    buf, desc = pool(L, c)
    append(L, c, desc, 0, n, True, True, True)
    assert L.dsv4sa_check_errors() == (0, 0)
    again, adesc = pool(L, c)
    start = again.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        append(L, c, adesc, 0, n, True, True, True)
    for _ in range(2):
        again.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, buf)
