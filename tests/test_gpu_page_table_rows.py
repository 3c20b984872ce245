"""Rows of a page table that a call's lists name but the table does not have.  The tables here are the
first rows of larger ones whose other rows hold good pages, so that a row behind the table would be
read without a fault, and show."""
import numpy as np
import pytest
import torch

from test_gpu_kv_fp4 import dev
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
