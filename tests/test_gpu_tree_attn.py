"""Attention of drafted tokens on the GPU against fp64.

Tolerance, as derived for the 4-bit cache's attention (test_gpu_kv_fp4.py): the rows are the
BF16 values that the oracle takes too; P is rounded to BF16 (2^-8 of each probability), the
output as well (2^-8 of it), a score is an fp32 sum of 512 products (error at most eps_s = 512 *
2^-24 * scale * sum_d |q_d kv_jd|), which moves a probability by a factor e^eps_s:
  |err| <= (2^-8 + 2 eps_s + 2^-15) * A + 2^-8 |o|,  A = sum_j p_j |kv_jd| / Z
with 2^-15 for the fp32 sums over up to 20000 rows in pieces, the exponentials and the joining
of the pieces, and 2^-126 max |kv| for each row that fp32 flushes to zero.
|lse err| <= eps_s + 2^-15 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv_fp4 import bf16_dev, bits_of, dev, random_pool

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def make_pool(rng, kind, P):
    if kind == 3:
        return random_pool(rng, P, 124, 129)
    x = rng.standard_normal((P, 64, 7, 64)).astype(np.float32)
    scale = (np.maximum(np.abs(x).max(-1), 1e-4) / np.float32(448)).astype(np.float32)
    codes = torch.from_numpy(x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return {"nope_codes": codes.reshape(P, 64, 448), "nope_scale": scale, "rope_bits": bits_of(rng.standard_normal((P, 64, 64)))}


def pack(L, kind, p):
    if kind == 3:
        return L.pack_kv_pool_fp4(p["nope_codes"], p["nope_e8m0"], p["rope_bits"])
    return L.pack_kv_pool(p["nope_codes"], p["nope_scale"], p["rope_bits"])


def rows_of(kind, pool, pt_row, entries):
    """The rows as the attention reads them: BF16 values."""
    e = np.asarray(entries, np.int64)
    if e.size == 0:
        return np.zeros((0, 512))
    if kind == 3:
        return oracle.kv_rows_fp4(pool, pt_row, e)
    v = oracle.kv_rows(pool, pt_row, e)
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()


class Batch:
    """Trees over random pools.  seqs: (committed tokens, parents of its nodes, entries) each."""

    def __init__(self, L, seqs, H, kind=0, window=128, ring=128, draft=128, ratio=128, seed=0, behind=0, sharp=1.0, chain=False):
        rng = np.random.default_rng(seed)
        self.L, self.kind, self.H, self.window, self.ring, self.draft, self.chain = L, kind, H, window, ring, draft, chain
        B = len(seqs)
        self.start = np.concatenate([[0], np.cumsum([len(p) for _, p, _ in seqs])]).astype(np.int32)
        self.T = int(self.start[-1]) + behind
        self.ctx = np.array([c for c, _, _ in seqs], np.int32)
        pos, anc, nv = [], [], []
        for c, parents, entries in seqs:
            masks = oracle.tree_masks(parents)
            p = [c + bin(m).count("1") - 1 for m in masks]
            pos += p
            anc += masks
            nv += [min((x + 1) // ratio, entries) for x in p]
        self.pos = np.array(pos + [0] * behind, np.int32)
        self.anc = np.array(anc + [0] * behind, np.uint64)
        self.n_vis = np.array(nv + [0] * behind, np.int32)
        self.n_max = max([e for _, _, e in seqs] + [0])
        per, wper = max(1, -(-self.n_max // 64)), max(1, -(-((ring if ring else int(self.ctx.max(initial=0))) + 0) // 64)) + 1
        if ring == 0:
            wper = max(1, -(-int(self.ctx.max(initial=1)) // 64)) + 2
        if draft >= 0:
            wper = max(wper, -(-(draft + 64) // 64))
        self.comp, self.win = make_pool(rng, kind, B * per + 1), make_pool(rng, kind, B * wper + 1)
        self.comp_pt = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        self.win_pt = rng.permutation(B * wper + 1)[:B * wper].reshape(B, wper).astype(np.int32)
        self.seq_row = rng.permutation(B).astype(np.int32)
        self.q = bits_of(sharp * rng.standard_normal((max(self.T, 1), H, 512)))
        self.sink = rng.standard_normal(H).astype(np.float32)
        self.max_nodes = max([len(p) for _, p, _ in seqs] + [1])
        self.rope = None

    def upload(self):
        L = self.L
        self.comp_buf, self.comp_desc = pack(L, self.kind, self.comp)
        self.win_buf, self.win_desc = pack(L, self.kind, self.win)
        self.dev = {n: dev(getattr(self, n)) for n in ("start", "ctx", "pos", "n_vis", "comp_pt", "win_pt", "seq_row", "sink")}
        self.dev["anc"] = dev(self.anc.view(np.int64))
        self.dev["q"] = bf16_dev(self.q)
        n = L.dsv4sa_tree_attn_workspace_size(len(self.ctx), self.max_nodes, self.H, self.n_max, self.window)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.out = torch.full(self.dev["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full(self.dev["q"].shape[:2], 7.0, device="cuda")

    def call(self, stream=None, out=None, lse=None, ws=None):
        d = self.dev
        rope = {} if self.rope is None else dict(rope_cs=self.rope[0], rope_pos=self.rope[1])
        self.L.dsv4sa_tree_attn(d["q"], d["sink"], d["start"], d["ctx"], d["pos"], self.comp_desc if self.n_max else None, d["comp_pt"],
                                d["n_vis"], self.n_max, self.win_desc, d["win_pt"], self.window, self.out if out is None else out, SCALE,
                                max_nodes=self.max_nodes, seq_row=d["seq_row"], anc=None if self.chain else d["anc"],
                                win_ring=self.ring, draft_entry=self.draft, lse=self.lse if lse is None else lse,
                                ws=self.ws if ws is None else ws, stream=stream, **rope)

    def nodes(self):
        for b in range(len(self.ctx)):
            for t in range(self.start[b], self.start[b + 1]):
                yield b, t

    def rows(self, b, t):
        r = self.seq_row[b]
        n = int(self.start[b + 1] - self.start[b])
        mask = (2 << int(t - self.start[b])) - 1 if self.chain else int(self.anc[t])
        win, drafts = oracle.tree_window(int(self.pos[t]), int(self.ctx[b]), self.window, self.ring, mask, n, self.draft)
        e = np.concatenate([win[win >= 0], drafts[drafts >= 0]])
        return np.concatenate([rows_of(self.kind, self.comp, self.comp_pt[r], np.arange(max(0, min(int(self.n_vis[t]), self.n_max)))),
                               rows_of(self.kind, self.win, self.win_pt[r], e)])

    def check_node(self, b, t, rotate=None):
        rows, q = self.rows(b, t), oracle.bf16_decode(self.q[t])
        want, lse = oracle.sink_softmax_attention(q, rows, self.sink, SCALE), oracle.attend_lse(q, rows, self.sink, SCALE)
        got, glse = self.out[t].double().cpu().numpy(), self.lse[t].double().cpu().numpy()
        if rows.shape[0] == 0:
            assert (got == 0).all()
            np.testing.assert_allclose(glse, self.sink, rtol=2.0 ** -20, atol=2.0 ** -20)
            return
        eps = (512 * 2.0 ** -24 * SCALE * (np.abs(q) @ np.abs(rows).T)).max(axis=1)           # [H]
        p = np.exp(SCALE * (q @ rows.T) - lse[:, None])
        A = p @ np.abs(rows)
        bound = (2.0 ** -8 + 2 * eps + 2.0 ** -15)[:, None] * A + rows.shape[0] * 2.0 ** -126 * np.abs(rows).max()
        if rotate is not None:
            want = rotate(want)
            pair = bound[:, 448:].reshape(self.H, 32, 2).sum(2)
            bound[:, 448:] = np.repeat(pair, 2, axis=1) + 2.0 ** -20 * np.repeat(np.abs(want[:, 448:]).reshape(self.H, 32, 2).sum(2), 2, axis=1)
        over = np.abs(got - want) - bound - 2.0 ** -8 * np.abs(want)
        assert over.max() <= 0, (b, t, over.max())
        assert (np.abs(glse - lse) <= eps + 2.0 ** -15 + 2.0 ** -22 * np.abs(lse)).all(), (b, t)

    def run_and_check(self, only=None):
        self.upload()
        self.call()
        assert self.L.dsv4sa_check_errors() == (0, 0)
        todo = list(self.nodes())
        for b, t in todo if only is None else [todo[i] for i in only]:
            self.check_node(b, t)
        assert (self.out[int(self.start[-1]):] == 7).all() and (self.lse[int(self.start[-1]):] == 7).all()


def chain(n):
    return list(range(-1, n - 1))


def tree(rng, n):
    return [-1] + [int(rng.integers(-1, j)) for j in range(1, n)]


RNG = np.random.default_rng(5)


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("seqs,H", [
    ([(0, [-1], 0)], 1), ([(5, [-1], 0)], 16), ([(700, [-1], 5)], 64), ([(129, chain(3), 1)], 128), ([(64, tree(RNG, 64), 0)], 1),
    ([(1000, tree(RNG, 13), 7), (0, [], 0), (3, tree(RNG, 64), 0), (128 * 40, chain(5), 40)], 8),
    ([(128 * 300 + 77, tree(RNG, 9), 300), (128 * 11, [-1], 11), (17, chain(2), 0)], 65),
    ([(256, tree(RNG, 6), 2)] * 40, 3)])
def test_trees_match_oracle(L, seqs, H, kind):
    Batch(L, seqs, H, kind, seed=len(seqs) * 100 + H, behind=2).run_and_check()


@pytest.mark.parametrize("window,ring,draft", [(0, 0, 5), (1, 1, 64), (60, 64, 64), (128, 0, 700), (200, 256, 300), (128, 128, -1), (0, 0, -1)])
def test_windows(L, window, ring, draft):
    seqs = [(600, tree(RNG, 7), 4), (30, chain(4), 0), (0, tree(RNG, 3), 0), (128, [-1], 1)]
    Batch(L, seqs, 24, 0, window=window, ring=ring, draft=draft, seed=window + 1).run_and_check()


def test_only_entries(L):
    b = Batch(L, [(128 * 70, [-1, -1], 70), (128 * 3, [-1], 3)], 64, 0, window=0, ring=0, draft=-1, seed=4)
    b.run_and_check()


def test_chain_is_the_default(L):
    b = Batch(L, [(300, chain(9), 2), (5, chain(64), 0)], 5, 3, seed=6, chain=True)
    b.run_and_check()


@pytest.mark.parametrize("kind,n", [(0, 20011), (3, 8192)])
def test_long_sequences(L, kind, n):
    """One sequence over the whole GPU, its rows cut into one piece for each CTA."""
    b = Batch(L, [(128 * n + 5, tree(RNG, 3), n)], 64, kind, seed=n)
    b.run_and_check()
    c = Batch(L, [(128 * n, [-1], n), (5, [-1], 0)], 4, kind, seed=n + 1, sharp=4.0)
    c.run_and_check()


def test_sharp_scores_and_late_maxima(L):
    """Scores far apart, the largest in the last rows: the max in use moves and sums are rescaled."""
    b = Batch(L, [(128 * 1000, chain(2), 1000), (128 * 5, tree(RNG, 5), 5)], 64, 0, seed=9, sharp=16.0)
    q = oracle.bf16_decode(b.q[0])
    b.win["rope_bits"][b.win_pt[b.seq_row[0]], :] = bits_of(q[3, 448:] * 4)      # one head's query in the window's rows
    b.run_and_check()


def test_every_node_of_a_large_batch(L):
    rng = np.random.default_rng(10)
    seqs = [(int(rng.integers(0, 128 * 600)), tree(rng, int(rng.integers(1, 17))), 600) for _ in range(24)]
    b = Batch(L, seqs, 64, 0, seed=11)
    b.run_and_check(only=range(0, int(b.start[-1]), 7))


def test_nodes_that_see_nothing(L):
    b = Batch(L, [(0, [-1, 0, -1], 0), (128 * 4, [-1, 0, 1], 4), (0, [-1], 0)], 16, 0, seed=12)
    b.anc[0] = b.anc[2] = b.anc[6] = 0
    b.anc[4] = 0
    b.n_vis[4] = -3
    b.pos[4] = -9
    b.run_and_check()
    assert (b.out[0] == 0).all() and (b.out[4] == 0).all() and (b.out[6] == 0).all()
    b.sink[:] = -np.inf
    b.upload()
    b.call()
    assert (b.out[6] == 0).all() and torch.isneginf(b.lse[6]).all()


def test_bits_above_the_nodes_and_masks_with_holes(L):
    b = Batch(L, [(10, chain(3), 0), (300, chain(6), 2)], 32, 0, seed=13)
    b.anc[:] |= np.uint64(0xFFFF_FFFF_FFFF_FF00)
    b.anc[5] = np.uint64(0b100001)
    b.upload()
    b.call()
    for bb, t in b.nodes():
        keep = b.anc[t]
        b.anc[t] = keep & np.uint64((1 << int(b.start[bb + 1] - b.start[bb])) - 1)
        b.check_node(bb, t)
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("what", ["nan", "inf", "scale"])
def test_a_bad_row_reaches_its_own_nodes_only(L, kind, what):
    """H = 4: all nodes of a sequence share an item.  Drafted row 2 and the last entry hold no numbers."""
    parents = [-1, 0, 0, 2, 1]                        # nodes 2 and 3 see row 2
    b = Batch(L, [(128 * 200 + 126, parents, 201), (128 * 3, chain(2), 3)], 4, kind, seed=14)
    assert b.n_vis[:5].tolist() == [200, 201, 201, 201, 201]
    row, last = b.seq_row[0], 200

    def spoil(pool, pt, e):
        pg, sl = pt[row, e // 64], e % 64
        if what == "scale":
            if kind == 3:
                pool["nope_e8m0"][pg, sl, 3] = 255
            else:
                pool["nope_scale"][pg, sl, 3] = np.inf
        else:
            pool["rope_bits"][pg, sl, 9] = 0x7FC0 if what == "nan" else 0xFF80
    spoil(b.win, b.win_pt, 128 + 2)
    b.upload()
    b.call()
    got = b.out.float().cpu()
    for bb, t in b.nodes():
        if bb == 0 and t in (2, 3):
            assert got[t].isnan().all() and b.lse[t].isnan().all()
        else:
            b.check_node(bb, t)
    spoil(b.comp, b.comp_pt, last)                    # all but node 0 see the last entry
    b.upload()
    b.call()
    got = b.out.float().cpu()
    for bb, t in b.nodes():
        if bb == 0 and t > 0:
            assert got[t].isnan().all()
        else:
            b.check_node(bb, t)
    assert L.dsv4sa_check_errors() == (0, 0)


def test_a_bad_query_stays_alone(L):
    b = Batch(L, [(128 * 20, [-1, 0, 0, 1], 20)], 16, 0, seed=15)
    b.q[1, :, 7] = 0x7FC0
    b.q[2, 5, 9] = 0x7F80
    b.upload()
    b.call()
    for bb, t in b.nodes():
        if t == 1:
            assert b.out[t].isnan().all()
        elif t != 2:
            b.check_node(bb, t)
    heads = [h for h in range(16) if h != 5]
    b.q[2, 5] = 0
    ref = oracle.sink_softmax_attention(oracle.bf16_decode(b.q[2]), b.rows(0, 2), b.sink, SCALE)[heads]
    assert np.abs(b.out[2].double().cpu().numpy()[heads] - ref).max() < 0.05


def test_pages_out_of_range_take_out_their_rows(L):
    b = Batch(L, [(128 * 200, chain(3), 200), (128 * 3, chain(2), 3)], 64, 0, seed=16)
    b.upload()
    pt = b.comp_pt.copy()
    pt[b.seq_row[0], 1] = -1
    pt[b.seq_row[0], 2] = 10 ** 6
    b.dev["comp_pt"].copy_(torch.from_numpy(pt))
    b.call()
    assert L.dsv4sa_check_errors() == (5, 1)
    r = b.seq_row[0]
    keep = [e for e in range(200) if not 64 <= e < 192]
    for t in range(3):
        win, drafts = oracle.tree_window(int(b.pos[t]), int(b.ctx[0]), 128, 128, (2 << t) - 1, 3, 128)
        e = np.concatenate([win[win >= 0], drafts[drafts >= 0]])
        rows = np.concatenate([rows_of(0, b.comp, b.comp_pt[r], keep), rows_of(0, b.win, b.win_pt[r], e)])
        ref = oracle.sink_softmax_attention(oracle.bf16_decode(b.q[t]), rows, b.sink, SCALE)
        assert np.abs(b.out[t].double().cpu().numpy() - ref).max() <= 2e-2
    for t in (3, 4):
        b.check_node(1, t)


def test_bounds_that_are_no_sequence(L):
    b = Batch(L, [(128 * 2, chain(4), 2), (50, chain(3), 0), (128, chain(2), 1), (9, [-1], 0)], 16, 0, seed=17)
    for bad in ([0, 4, 2, 9, 10], [0, 4, 7, 9, 12], [0, 9, 7, 9, 10], [-3, 4, 7, 9, 10]):
        b.upload()
        b.dev["start"].copy_(torch.tensor(bad, dtype=torch.int32))
        b.call()
        assert L.dsv4sa_check_errors() == (5, 1)
        covered = np.zeros(b.T, bool)
        for s in range(4):
            lo, hi = bad[s], bad[s + 1]
            if 0 <= lo <= hi <= b.T and hi - lo <= b.max_nodes:
                covered[lo:hi] = True
        out = b.out.float().cpu().numpy()
        assert (out[~covered] == 7).all() and (out[covered] != 7).any(axis=(1, 2)).all()


@pytest.mark.parametrize("n", [3, 400])
def test_rotated_output(L, n):
    rng = np.random.default_rng(18)
    b = Batch(L, [(128 * n + 9, tree(rng, 5), n), (40, chain(3), 0)], 48, 0, seed=19)
    cs = torch.empty(1000, 32, 2, device="cuda")
    L.dsv4sa_rope_table(cs, base=160000.0)
    pos = rng.integers(0, 1000, b.T).astype(np.int32)
    b.rope = (cs, dev(pos))
    b.upload()
    b.call()
    assert L.dsv4sa_check_errors() == (0, 0)
    z = cs.double().cpu().numpy()
    z = z[..., 0] + 1j * z[..., 1]
    for bb, t in b.nodes():
        b.check_node(bb, t, rotate=lambda o, t=t: oracle.rotate_heads(o, z[pos[t]], 448, False, inverse=True))
    pos[1] = 1000
    plain = Batch(L, [(128 * n + 9, tree(np.random.default_rng(18), 5), n), (40, chain(3), 0)], 48, 0, seed=19)
    plain.upload()
    plain.call()
    b.rope = (cs, dev(pos))
    b.call()
    assert L.dsv4sa_check_errors() == (5, 1)
    assert torch.equal(b.out[1], plain.out[1]) and not torch.equal(b.out[0], plain.out[0])


def test_same_bits_again_in_graphs_and_on_streams(L):
    """Two graphs that share a workspace, replayed in turn; a call on another stream; no lse."""
    a = Batch(L, [(128 * 900, tree(RNG, 4), 900), (128 * 30, chain(3), 30)], 64, 0, seed=20)
    c = Batch(L, [(128 * 50, chain(2), 50)], 16, 0, seed=21)
    a.upload()
    c.upload()
    ws = a.ws if a.ws.numel() >= c.ws.numel() else c.ws
    refs = []
    for x in (a, c):
        x.call(ws=ws)
        refs.append((x.out.clone(), x.lse.clone()))
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for x in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.call(ws=ws)
        graphs.append(g)
    for _ in range(3):
        for x, g, (out, lse) in zip((a, c), graphs, refs):
            x.out.zero_(), x.lse.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(x.out, out) and torch.equal(x.lse, lse)
    a.out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    a.call(stream=s, ws=ws)
    s.synchronize()
    assert torch.equal(a.out, refs[0][0])
    d = c.dev
    L.dsv4sa_tree_attn(d["q"], d["sink"], d["start"], d["ctx"], d["pos"], c.comp_desc, d["comp_pt"], d["n_vis"], c.n_max, c.win_desc,
                       d["win_pt"], c.window, c.out, SCALE, max_nodes=c.max_nodes, seq_row=d["seq_row"], win_ring=128,
                       draft_entry=128, ws=ws)
    assert torch.equal(c.out, refs[1][0])             # its masks are a chain's
    assert L.dsv4sa_check_errors() == (0, 0)


def test_no_sequences(L):
    b = Batch(L, [(9, [-1], 0)], 16, 0, seed=22)
    b.upload()
    d = b.dev
    for start, q, nodes in ((d["start"][:1], d["q"], 1), (d["start"], d["q"][:0], 1), (d["start"], d["q"], 0)):
        out = torch.full_like(q, 7.0)
        L.dsv4sa_tree_attn(q, d["sink"], start, d["ctx"], d["pos"], None, None, d["n_vis"], 0, b.win_desc, d["win_pt"], 128, out, SCALE,
                           max_nodes=nodes, win_ring=128, draft_entry=128)
        assert (out == 7).all()
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("window,ring,draft", [(128, 128, 128), (1, 0, 9), (0, 0, 3), (60, 64, -1)])
def test_window_lists(L, window, ring, draft):
    b = Batch(L, [(600, tree(RNG, 7), 4), (0, [], 0), (30, chain(4), 0), (0, tree(RNG, 3), 0)], 16, 0, window=window, ring=ring,
              draft=draft, seed=30, behind=2)
    b.upload()
    m = b.max_nodes
    for chained in (False, True):
        idx = torch.full((b.T, window + m + 3), -7, dtype=torch.int32, device="cuda")
        L.dsv4sa_tree_window_indices(b.dev["start"], b.dev["ctx"], b.dev["pos"], window, ring, draft, m, idx,
                                     anc=None if chained else b.dev["anc"])
        got = idx.cpu().numpy()
        want = np.full_like(got, -7)
        for s, t in b.nodes():
            n = int(b.start[s + 1] - b.start[s])
            mask = (2 << int(t - b.start[s])) - 1 if chained else int(b.anc[t])
            win, drafts = oracle.tree_window(int(b.pos[t]), int(b.ctx[s]), window, ring, mask, n, draft)
            want[t, :window + m] = -1
            want[t, :window] = win
            want[t, window:window + n] = drafts
        np.testing.assert_array_equal(got, want)
    assert L.dsv4sa_check_errors() == (0, 0)
    L.dsv4sa_tree_window_indices(torch.tensor([0, 99], dtype=torch.int32, device="cuda"), b.dev["ctx"], b.dev["pos"], window, ring, draft, m, idx)
    assert L.dsv4sa_check_errors() == (5, 1)


def test_lists_and_trees_agree(L):
    """The sparse attention over all entries and a node's window list, against the tree attention."""
    b = Batch(L, [(128 * 40 + 5, tree(RNG, 9), 40), (70, chain(3), 0)], 64, 0, seed=31)
    b.upload()
    b.call()
    kw = 128 + b.max_nodes
    idx_w = torch.empty(b.T, kw, dtype=torch.int32, device="cuda")
    idx_c = torch.empty(b.T, b.n_max, dtype=torch.int32, device="cuda")
    d = b.dev
    L.dsv4sa_tree_window_indices(d["start"], d["ctx"], d["pos"], 128, 128, 128, b.max_nodes, idx_w, anc=d["anc"])
    L.dsv4sa_compress_indices(d["n_vis"], b.n_max, idx_c)
    q_seq = d["seq_row"][torch.tensor([0] * 9 + [1] * 3, device="cuda")].contiguous()
    out, lse = torch.empty_like(b.out), torch.empty_like(b.lse)
    ws = torch.empty(L.dsv4sa_attn_workspace_size(L.ATTN_DECODE, b.T, 64, b.n_max, kw), dtype=torch.uint8, device="cuda")
    L.dsv4sa_sparse_attn_decode(d["q"], d["sink"], q_seq, b.comp_desc, d["comp_pt"], idx_c, b.win_desc, d["win_pt"], idx_w, out, SCALE,
                                lse=lse, ws=ws)
    assert L.dsv4sa_check_errors() == (0, 0)
    # the sparse attention's own tolerance (it merges its splits in BF16)
    assert (b.out.float() - out.float()).abs().max() <= 2e-2
    assert (lse - b.lse).abs().max() <= 1e-3
