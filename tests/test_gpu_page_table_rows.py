"""Rows of a page table that a call's lists name but the table does not have.  The tables here are the
first rows of larger ones whose other rows hold good pages, so that a row behind the table would be
read without a fault, and show."""
import numpy as np
import pytest
import torch

from test_gpu_append import device_pool, fp8_pool, table_of
from test_gpu_kv_fp4 import bf16_dev, bits_of, dev, random_pool
from test_gpu_tree_attn import Batch, chain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def first_rows(pt, more=2):
    """pt on the device, `more` copies of its rows behind it in the same allocation."""
    return torch.from_numpy(np.concatenate([pt] * (more + 1))).cuda()[:pt.shape[0]]


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("row", [3, 4, 8, -1])
def test_tree_attention(L, kind, row):
    """Sequence 1's row is none of the table's three."""
    b = Batch(L, [(128 * 5, chain(2), 5), (128 * 130 + 3, [-1, 0, 0], 130), (40, [-1], 0)], 16, kind, seed=41)
    b.upload()
    b.dev["comp_pt"], b.dev["win_pt"] = first_rows(b.comp_pt), first_rows(b.win_pt)
    rows = b.seq_row.copy()
    rows[1] = row
    b.dev["seq_row"] = dev(rows)
    b.call()
    assert L.dsv4sa_check_errors() == (5, 1)
    for s, t in b.nodes():
        if s != 1:
            b.check_node(s, t)
            continue
        assert (b.out[t] == 0).all()                 # no row is left: the sink alone
        np.testing.assert_allclose(b.lse[t].double().cpu().numpy(), b.sink, rtol=2.0 ** -20, atol=2.0 ** -20)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kind", [0, 3])
def test_appended_rows(L, kind, norm):
    """Rows 1 and 3 name a row that the table does not have: neither is written, the others are."""
    rng = np.random.default_rng(42)
    pool = fp8_pool(rng, 8) if kind == L.POOL_KV else random_pool(rng, 8)
    pt = rng.permutation(8).reshape(2, 4).astype(np.int32)
    cs, _ = table_of(L, 50)
    rows = bf16_dev(bits_of(rng.standard_normal((5, 512))))
    eps = 1e-6 if norm else None
    seq, pos = np.array([0, 2, 1, 5, 0], np.int32), np.array([3, 4, 5, 6, 7], np.int32)
    buf, desc = device_pool(L, kind, pool)
    L.dsv4sa_cache_append(desc, first_rows(pt), dev(seq), dev(pos), rows, cs, eps=eps)
    assert L.dsv4sa_check_errors() == (5, 1)
    want, wdesc = device_pool(L, kind, pool)
    L.dsv4sa_cache_append(wdesc, dev(pt), dev(np.where(seq < 2, seq, -1).astype(np.int32)), dev(pos), rows, cs, eps=eps)
    assert L.dsv4sa_check_errors() == (0, 0)
    assert torch.equal(buf, want)
