"""ATTN_EARLY_WINDOW over FP4 pools gives the bits of the call without it, whatever the split
over heads and clusters and wherever a query lies in its CTA's work."""
import os

import numpy as np
import pytest
import torch

from test_gpu_kv_fp4 import SCALE, Case, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


# lists whose window fills chunks, ends inside one, makes one more chunk or none; no window; no list
@pytest.mark.parametrize("T,H,kc,kw,ring", [(1, 16, 512, 128, 128), (1, 64, 512, 128, 128), (8, 64, 500, 100, 128), (32, 64, 512, 128, 128),
                                            (32, 64, 600, 60, 64), (3, 40, 2048, 1000, 1024), (16, 64, 96, 33, 64), (5, 64, 129, 127, 128),
                                            (2, 16, 100, 28, 64), (130, 64, 700, 200, 256), (400, 80, 150, 32, 64), (200, 20, 300, 129, 192),
                                            (4, 24, 0, 130, 192), (4, 24, 300, 0, 0), (64, 16, 1000, 128, 0)])
def test_the_flag_changes_no_bit(L, T, H, kc, kw, ring):
    c = Case(L, T, H, kc, kw, seed=T + 3 * H + kc + kw, ring=ring, entries=3000 if kc > 1500 else 1500, empty=(0, T - 1) if T > 5 else ())
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        plain, early = c.run(L, fn), c.run(L, fn, flags=L.ATTN_EARLY_WINDOW)
        assert same(plain, early)
        assert same(plain, c.run(L, fn, explicit=True, flags=L.ATTN_EARLY_WINDOW))
        c.check(*early, rows=sorted({0, 1 % T, T // 2, T - 1}))
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("T,H,k", [(32, 64, 512), (10, 16, 300), (160, 64, 512)])
def test_the_flag_behind_the_selection_that_it_overlaps(L, T, H, k):
    """The top-k writes the lists while the window's rows are already worked on."""
    c = Case(L, T, H, k, 100, seed=T, ring=128)
    N = c.comp_pt.shape[1] * 64
    logits = torch.randn(T, N, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    n_vis = torch.randint(0, N + 1, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    d, got = c.d, []
    for flags in (0, L.ATTN_EARLY_WINDOW):
        for fused in (False, True):
            idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
            out, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
            args = (d["q"], d["sink"], d["seq"], c.comp_d, d["comp_pt"], idx, c.win_d, d["win_pt"], None, out, SCALE)
            kw = dict(lse=lse, win_pos=d["pos"], kw=100, win_ring=128, flags=flags)
            if fused:
                L.dsv4sa_topk_sparse_attn_decode(logits, n_vis, N, k, *args, **kw)
            else:
                L.dsv4sa_topk(logits, n_vis, N, k, idx)
                L.dsv4sa_sparse_attn_decode(*args, **kw)
            got.append((out, lse, idx))
    for other in got[1:]:
        assert same(got[0], other) and torch.equal(got[0][2], other[2])
    c.idx = got[0][2].cpu().numpy()
    c.check(*got[0][:2], rows=[0, T // 2, T - 1])
    assert L.dsv4sa_check_errors() == (0, 0)


def test_a_query_keeps_its_bits_when_the_others_change(L):
    """At a given number of queries a query's result does not depend on the others' vectors,
    lists and windows: clusters (32 queries), and several items a CTA (400)."""
    for T, H in ((32, 64), (400, 80)):
        c = Case(L, T, H, 300, 128, seed=T, ring=128)
        for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
            before = c.run(L, fn)
            keep = np.arange(T) % 3 == 1
            q, idx, pos = c.d["q"].clone(), c.d["idx"].clone(), c.d["pos"].clone()
            away = dev(~keep)
            c.d["q"][away] = 4 * c.d["q"][away].flip(1)
            c.d["idx"][away] = torch.where(c.d["idx"][away] >= 0, (c.d["idx"][away] * 7 + 3) % 1500, -1)
            c.d["idx"][dev(np.arange(T) % 6 == 0)] = -1
            c.d["pos"][away] = (c.d["pos"][away] * 5 + 1) % 640
            after = c.run(L, fn)
            stay = dev(keep)
            assert same([t[stay] for t in before], [t[stay] for t in after])
            assert not torch.equal(before[0][away], after[0][away])
            c.d["q"], c.d["idx"], c.d["pos"] = q, idx, pos
    assert L.dsv4sa_check_errors() == (0, 0)
