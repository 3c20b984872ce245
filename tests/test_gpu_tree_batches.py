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


def test_most_sequences(L):
    """2^24 sequences, all but two of them empty, the long one's item cut: a CTA has its end and, far behind it, the last item."""
    b = Batch(L, [(128 * 4000, chain(3), 4000), (200, chain(2), 1)], 16, 0, seed=43)
    n = 2 ** 24
    b.upload()
    start = torch.full((n + 1,), 3, dtype=torch.int32, device="cuda")
    start[0], start[n] = 0, 5
    ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
    ctx[0], ctx[n - 1] = int(b.ctx[0]), int(b.ctx[1])
    row = torch.full((n,), 10 ** 6, dtype=torch.int32, device="cuda")
    row[0], row[n - 1] = int(b.seq_row[0]), int(b.seq_row[1])
    b.dev.update(start=start, ctx=ctx, seq_row=row)
    b.ws = torch.empty(L.dsv4sa_tree_attn_workspace_size(n, b.max_nodes, 16, b.n_max, b.window), dtype=torch.uint8, device="cuda")
    b.call()
    assert L.dsv4sa_check_errors() == (0, 0)
    for s, t in b.nodes():
        b.check_node(s, t)


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("n", [897, 1800])
def test_more_sequences_than_threads(L, n, kind):
    """A thread of the scan counts several items: short sequences, a third of them empty, and two longer ones.  There
    are more items than CTAs, so some are cut."""
    rng = np.random.default_rng(n)
    seqs = [(int(rng.integers(0, 600)), tree(rng, int(rng.integers(0, 3))) if i % 3 else [], 4) for i in range(n)]
    seqs[n // 2] = (128 * 250 + 7, chain(5), 250)
    seqs[-1] = (128 * 200, tree(rng, 4), 200)
    b = Batch(L, seqs, 16, kind, seed=n)
    t = int(b.start[n // 2])
    some = sorted(set(range(0, b.T, 97)) | set(range(t - 3, t + 8)) | {b.T - 1})
    b.run_and_check(some)
    out, lse = b.out.clone(), b.lse.clone()
    b.call()
    assert torch.equal(out, b.out) and torch.equal(lse, b.lse)


@pytest.mark.parametrize("n", [8, 16])
def test_items_left_whole_with_several_a_thread(L, n):
    """128 items a sequence at most (64 nodes of 128 heads) and one or two nodes in each: more places than threads, fewer items than CTAs."""
    rng = np.random.default_rng(n)
    seqs = [(int(rng.integers(0, 900)), chain(1 + i % 2) if i % 5 else [], 6) for i in range(n)]
    b = Batch(L, seqs, 128, 0, seed=n)
    b.max_nodes = 64
    b.run_and_check()


@pytest.mark.parametrize("empty", ["first", "last", "all but one"])
def test_threads_without_an_item(L, empty):
    n = 2000
    seqs = [(100, [-1], 0)] * n
    for i in range(n):
        if (empty == "first" and i < 1500) or (empty == "last" and i >= 500) or (empty == "all but one" and i != 1234):
            seqs[i] = (100, [], 0)
    b = Batch(L, seqs, 8, 0, seed=45)
    b.run_and_check(range(0, b.T, max(1, b.T // 40)))
