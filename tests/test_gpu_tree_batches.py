"""Attention of drafted tokens over batches at the ends of what a call may hold.  Tolerances as in
test_gpu_tree_attn.py."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attn import Batch, chain, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.mark.parametrize("start,errors", [([0, 0, 0, 0], (0, 0)), ([5, 5, 5, 5], (0, 0)), ([6, 5, 4, 3], (5, 1)), ([0, 6, 0, 7], (5, 1))])
def test_batches_without_a_node(L, start, errors):
    """Sequences, and queries behind them, but no node: every bound empty, or none a sequence's."""
    b = Batch(L, [(300, chain(2), 2), (0, [-1], 0), (128 * 9, tree(np.random.default_rng(1), 4), 9)], 16, 0, seed=40)
    b.upload()
    b.dev["start"].copy_(torch.tensor(start, dtype=torch.int32))
    b.max_nodes = 5
    b.ws = torch.empty(L.dsv4sa_tree_attn_workspace_size(3, 5, 16, b.n_max, b.window), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        b.call()
        assert L.dsv4sa_check_errors() == errors
        assert (b.out == 7).all() and (b.lse == 7).all()
    b.dev["start"].copy_(torch.from_numpy(b.start))        # the next batch is as any other
    b.call()
    assert L.dsv4sa_check_errors() == (0, 0)
    for s, t in b.nodes():
        b.check_node(s, t)
