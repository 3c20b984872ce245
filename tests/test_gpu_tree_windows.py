"""Windows of drafted tokens that do not lie side by side: nodes dropped (position -1, 0), branches at
positions of their own, and pages that no node needs any more.  Tolerances as in test_gpu_tree_attn.py."""
import numpy as np
import pytest
import torch

from test_gpu_kv_fp4 import dev
from test_gpu_tree_attn import Batch, chain, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def without_unseen_pages(b):
    """The batch's tables with -1 in place of every page that holds no row of any node."""
    comp, win = np.full_like(b.comp_pt, -1), np.full_like(b.win_pt, -1)
    for s, t in b.nodes():
        r, n = b.seq_row[s], int(b.start[s + 1] - b.start[s])
        mask = (2 << int(t - b.start[s])) - 1 if b.chain else int(b.anc[t])
        p = np.arange(max(0, int(b.pos[t]) - b.window + 1), min(int(b.pos[t]) + 1, int(b.ctx[s])))
        e = np.concatenate([p % b.ring if b.ring else p, [b.draft + j for j in range(n) if mask >> j & 1 and b.draft >= 0]]).astype(int)
        for pg in set(e // 64):
            win[r, pg] = b.win_pt[r, pg]
        for pg in range(-(-min(int(b.n_vis[t]), b.n_max) // 64)):
            comp[r, pg] = b.comp_pt[r, pg]
    return comp, win


def run(b):
    b.upload()
    comp, win = without_unseen_pages(b)
    b.dev["comp_pt"], b.dev["win_pt"] = dev(comp), dev(win)
    b.call()
    assert b.L.dsv4sa_check_errors() == (0, 0)
    for s, t in b.nodes():
        b.check_node(s, t)


@pytest.mark.parametrize("H", [1, 8, 64])
@pytest.mark.parametrize("far", [-1, -2 ** 31, 0, 63, 2000])
def test_one_node_far_off(L, far, H):
    """Raw tokens by position, the pages behind the windows released."""
    b = Batch(L, [(20000, chain(6), 9), (300, chain(3), 2)], H, 0, ring=0, draft=20100, seed=50)
    b.pos[2] = far
    run(b)


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("window,H", [(1, 1), (60, 1), (128, 1), (128, 5), (300, 2)])
def test_nodes_scattered_over_the_context(L, window, H, kind):
    """Sixty-four nodes anywhere from before the first token to behind the last committed one."""
    rng = np.random.default_rng(window + H)
    b = Batch(L, [(9000, tree(rng, 64), 70), (0, tree(rng, 5), 0), (700, tree(rng, 40), 5)], H, kind, window=window, ring=0, draft=9200, seed=51)
    for s in range(3):
        a, e = b.start[s], b.start[s + 1]
        b.pos[a:e] = rng.integers(-50, int(b.ctx[s]) + 2 * window + 60, e - a)
        b.pos[a + 1] = b.pos[a]                        # the same position twice
    run(b)


@pytest.mark.parametrize("gap", [-1, 0, 1, 2])
def test_windows_that_just_touch(L, gap):
    """Two groups of nodes `window` (+ gap) apart, in order and reversed: one run of positions or two."""
    for flip in (1, -1):
        b = Batch(L, [(5000, chain(4), 3)], 4, 0, window=100, ring=0, draft=5100, seed=52)
        b.pos[:] = np.array([1000, 1001, 1101 + gap, 1102 + gap])[::flip]
        run(b)


def test_scattered_nodes_of_a_ring(L):
    b = Batch(L, [(3000, tree(np.random.default_rng(3), 20), 9)], 3, 0, window=64, ring=4096, draft=4096, seed=53)
    b.pos[:] = np.random.default_rng(4).integers(0, 3100, 20)
    run(b)


def test_drafted_rows_that_no_node_sees(L):
    """Drafted rows 0 and 1 on a page that is not there, and seen by none."""
    b = Batch(L, [(200, chain(40), 1), (90, chain(5), 0)], 2, 0, ring=128, draft=190, seed=54)
    b.anc[:40] &= np.uint64(2 ** 64 - 4)
    run(b)
    b.anc[40] &= np.uint64(0)
    b.anc[41] = 0b11                                   # seen again, and its page missing in sequence 1
    b.upload()
    comp, win = without_unseen_pages(b)
    win[b.seq_row[1], 190 // 64] = -1
    b.dev["comp_pt"], b.dev["win_pt"] = dev(comp), dev(win)
    b.call()
    assert L.dsv4sa_check_errors() == (5, 1)


def test_far_nodes_cost_no_more_rows(L):
    """A dropped node in a long context: the call takes about as long as without it (it read a million rows for it)."""
    times = []
    for far in (None, 0):
        b = Batch(L, [(128 * 64, chain(5), 64)], 4, 0, seed=55)
        b.ctx[:] = 2 ** 20
        b.pos[:] = 2 ** 20 + np.arange(5)
        if far is not None:
            b.pos[3] = far
        b.upload()
        b.call()
        assert L.dsv4sa_check_errors() == (0, 0)
        for s, t in b.nodes():
            b.check_node(s, t)
        b.call()
        a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            b.call()
        e.record()
        e.synchronize()
        times.append(a.elapsed_time(e))
    assert times[1] < 3 * times[0], times


def test_no_committed_token(L):
    """ctx of 0 and below: no window, whatever the positions."""
    b = Batch(L, [(1000, chain(4), 7), (300, chain(3), 2), (500, chain(2), 3)], 8, 0, ring=0, draft=1100, seed=56)
    b.ctx[:] = [-2 ** 31, -5, 0]
    b.pos[1], b.pos[5] = 2 ** 31 - 1, 0
    run(b)
