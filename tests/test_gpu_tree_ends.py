"""Calls at the ends of what the attention of drafted tokens allows.  Tolerances as in
test_gpu_tree_attn.py."""
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


def check(b, only=None):
    b.call()
    assert b.L.dsv4sa_check_errors() == (0, 0)
    todo = list(b.nodes())
    for s, t in todo if only is None else [todo[i] for i in only]:
        b.check_node(s, t)


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("H", [127, 128])
def test_most_nodes_and_heads(L, H, kind):
    rng = np.random.default_rng(H)
    b = Batch(L, [(128 * 700 + 60, tree(rng, 64), 700), (50, chain(64), 0), (128 * 4, [-1], 4)], H, kind, seed=60)
    b.upload()
    check(b, [0, 1, 13, 31, 62, 63, 64, 100, 127, 128])


def test_widest_window(L):
    """65536 tokens, of a ring and by position, all of them committed and not yet so many."""
    for ring in (65536, 0):
        b = Batch(L, [(70000, chain(3), 3), (65535, [-1, 0, 0], 0), (900, [-1], 1)], 8, 0, window=65536, ring=ring, draft=70016, seed=61)
        b.upload()
        check(b)


def test_entries_above_the_list_are_clamped(L):
    b = Batch(L, [(128 * 90, chain(3), 90), (128 * 7, [-1, -1], 7)], 16, 0, seed=62)
    b.n_vis[1], b.n_vis[4] = 2 ** 31 - 1, 91
    b.upload()
    check(b)


def test_sequences_that_share_a_table_row(L):
    """Two sequences of one prefix: the same entries, ring and drafted rows, nodes of their own."""
    b = Batch(L, [(128 * 30 + 4, chain(4), 30), (128 * 30 + 4, tree(np.random.default_rng(2), 6), 30), (70, chain(2), 0)], 24, 3, seed=63)
    b.seq_row[1] = b.seq_row[0]
    b.upload()
    check(b)


def test_one_pool_for_entries_and_tokens(L):
    b = Batch(L, [(128 * 12 + 9, chain(3), 12), (200, tree(np.random.default_rng(3), 5), 1)], 16, 0, seed=64)
    pages = b.comp["nope_codes"].shape[0]
    both = {k: np.concatenate([b.comp[k], b.win[k]]) for k in b.comp}
    b.win_pt = (b.win_pt + pages).astype(np.int32)
    b.comp = b.win = both
    b.upload()
    b.win_desc = b.comp_desc
    check(b)


@pytest.mark.parametrize("scale", [0.0, -0.04, 3.0])
def test_scales(L, scale, monkeypatch):
    import test_gpu_tree_attn
    monkeypatch.setattr(test_gpu_tree_attn, "SCALE", scale)
    b = Batch(L, [(128 * 200, chain(3), 200), (60, [-1, -1], 0)], 16, 0, seed=65)
    b.upload()
    b.call()
    assert L.dsv4sa_check_errors() == (0, 0)
    import oracle
    for s, t in b.nodes():
        rows, q = b.rows(s, t), oracle.bf16_decode(b.q[t])
        want = oracle.sink_softmax_attention(q, rows, b.sink, scale)
        eps = (512 * 2.0 ** -24 * abs(scale) * (np.abs(q) @ np.abs(rows).T)).max(axis=1)
        p = np.exp(scale * (q @ rows.T) - oracle.attend_lse(q, rows, b.sink, scale)[:, None])
        bound = (2.0 ** -8 + 2 * eps + 2.0 ** -15)[:, None] * (p @ np.abs(rows)) + rows.shape[0] * 2.0 ** -126 * np.abs(rows).max()
        assert (np.abs(b.out[t].double().cpu().numpy() - want) <= bound + 2.0 ** -8 * np.abs(want)).all()


def test_calls_at_the_same_time(L):
    """Two streams, a workspace each, and appends and rotations on a third one: as one after the other."""
    a = Batch(L, [(128 * 2000, chain(4), 2000)], 64, 0, seed=66)
    c = Batch(L, [(128 * 50, chain(2), 50)] * 30, 16, 3, seed=67)
    refs = []
    for b in (a, c):
        b.upload()
        check(b, [0, 1])
        refs.append((b.out.clone(), b.lse.clone()))
    cs = torch.empty(100, 32, 2, device="cuda")
    L.dsv4sa_rope_table(cs)
    x = torch.randn(64, 8, 512, device="cuda").to(torch.bfloat16)
    pos = dev(np.arange(64, dtype=np.int32))
    want, got = torch.empty_like(x), torch.empty_like(x)
    L.dsv4sa_rope(x, cs, pos, out=want, eps=1e-6)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for b in (a, c):
            b.out.zero_(), b.lse.zero_()
        got.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            a.call(stream=streams[0])
            c.call(stream=streams[1])
            L.dsv4sa_rope(x, cs, pos, out=got, eps=1e-6, stream=streams[2])
        torch.cuda.synchronize()
        for b, (out, lse) in zip((a, c), refs):
            assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert L.dsv4sa_check_errors() == (0, 0)
