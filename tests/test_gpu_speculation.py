"""Steps of speculative decoding with the library's calls together: queries rotated, drafted rows
appended beside the ring, attention over the trees, the accepted path committed into the ring,
and the next token decoded from there -- against plain decoding one token at a time, where each
row enters the ring before its query attends (dsv4sa_sparse_attn_decode)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
H, WINDOW, DRAFT, RATIO = 16, 128, 128, 128


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Layer:
    """A layer without an indexer: ring and drafted rows of raw tokens, compressed entries, weights."""

    def __init__(self, L, kind, ctx, entries, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.L, self.B, self.kind = L, len(ctx), kind
        self.ctx, self.entries = list(ctx), entries
        self.g = g
        per, wper = -(-entries // 64), 3
        self.comp_buf, self.win_buf = L._alloc_pool(kind, self.B * per, "cuda"), L._alloc_pool(kind, self.B * wper, "cuda")
        self.comp, self.win = (L.dsv4sa_pool_desc_init(kind, b, n) for b, n in ((self.comp_buf, self.B * per), (self.win_buf, self.B * wper)))
        self.win_buf.zero_()
        self.comp_pt = torch.randperm(self.B * per, generator=g, device="cuda").view(self.B, per).to(torch.int32)
        self.win_pt = torch.randperm(self.B * wper, generator=g, device="cuda").view(self.B, wper).to(torch.int32)
        self.cs = torch.empty(4096, 32, 2, device="cuda")
        L.dsv4sa_rope_table(self.cs, base=160000.0, factor=4.0, original_len=1024)
        self.norm_w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
        self.sink = torch.randn(H, generator=g, device="cuda")
        n = self.B * entries
        seq = torch.arange(n, device="cuda") % self.B
        L.dsv4sa_cache_append(self.comp, self.comp_pt, seq.to(torch.int32), (torch.arange(n, device="cuda") // self.B).to(torch.int32),
                              self.rows(n))
        for b, c in enumerate(ctx):                  # the last tokens of the prompt, into the ring
            pos = np.arange(max(0, c - 128), c)
            if len(pos):
                self.commit([b] * len(pos), pos, self.rows(len(pos)))

    def rows(self, n):
        return torch.randn(n, 512, generator=self.g, device="cuda").to(torch.bfloat16)

    def commit(self, seq, pos, rows, src=None):
        self.L.dsv4sa_cache_append(self.win, self.win_pt, i32(seq), i32(pos), rows, self.cs, ring=128, norm_w=self.norm_w, eps=1e-6,
                                   src_row=src)

    def query(self, x, pos):
        q = torch.empty_like(x)
        self.L.dsv4sa_rope(x, self.cs, pos, out=q, eps=1e-6)
        return q

    def decode(self, b, pos, x, row):
        """One token in plain decoding: its row into the ring, then the sparse attention."""
        L = self.L
        self.commit([b], [pos], row)
        p = i32([pos])
        n_vis = min((pos + 1) // RATIO, self.entries)
        idx = torch.where(torch.arange(self.entries, device="cuda") < n_vis, torch.arange(self.entries, device="cuda"), -1).to(torch.int32)[None]
        out, lse = torch.empty(1, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, H, device="cuda")
        nb = L.dsv4sa_attn_workspace_size(L.ATTN_DECODE, 1, H, self.entries, WINDOW)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
        L.dsv4sa_sparse_attn_decode(self.query(x, p), self.sink, i32([b]), self.comp, self.comp_pt, idx.contiguous(), self.win, self.win_pt, None,
                                    out, SCALE, lse=lse, ws=ws, win_pos=p, kw=WINDOW, win_ring=128, rope_cs=self.cs, rope_pos=p)
        return out[0], lse[0]


@pytest.mark.parametrize("kind", [0, 3])
def test_drafts_accepted_and_decoded_on(L, kind):
    ctx = [700, 90, 0]
    spec, plain = (Layer(L, kind, ctx, 10, seed=5) for _ in range(2))
    rng = np.random.default_rng(1)
    for step in range(3):
        parents = [[-1, 0, 0, 1, 2, 2, 5], [-1, 0, 1], [-1, -1, 0, 1, 3]]
        masks = [oracle.tree_masks(p) for p in parents]
        start = np.concatenate([[0], np.cumsum([len(p) for p in parents])])
        T = int(start[-1])
        pos = np.array([c + bin(m).count("1") - 1 for c, ms in zip(spec.ctx, masks) for m in ms])
        seq = np.repeat(np.arange(3), np.diff(start))
        x = torch.randn(T, H, 512, generator=spec.g, device="cuda").to(torch.bfloat16)
        rows = spec.rows(T)
        plain.g.set_state(spec.g.get_state())
        out, lse = torch.empty_like(x), torch.empty(T, H, device="cuda")
        args = dict(start=i32(start), ctx=i32(spec.ctx), pos=i32(pos), seq=i32(seq), entry=i32(DRAFT + np.arange(T) - start[seq]),
                    n_vis=i32(np.minimum((pos + 1) // RATIO, 10)),
                    anc=torch.tensor([m for ms in masks for m in ms], dtype=torch.int64, device="cuda"),
                    ws=torch.empty(L.dsv4sa_tree_attn_workspace_size(3, 7, H, 10, WINDOW), dtype=torch.uint8, device="cuda"))

        def draft(q):
            L.dsv4sa_rope(x, spec.cs, args["pos"], out=q, eps=1e-6)
            L.dsv4sa_cache_append(spec.win, spec.win_pt, args["seq"], args["pos"], rows, spec.cs, row_entry=args["entry"],
                                  norm_w=spec.norm_w, eps=1e-6)
            L.dsv4sa_tree_attn(q, spec.sink, args["start"], args["ctx"], args["pos"], spec.comp, spec.comp_pt, args["n_vis"], 10, spec.win,
                               spec.win_pt, WINDOW, out, SCALE, max_nodes=7, anc=args["anc"], win_ring=128, draft_entry=DRAFT, lse=lse,
                               ws=args["ws"], rope_cs=spec.cs, rope_pos=args["pos"])
        q = torch.empty_like(x)
        draft(q)
        eager = out.clone(), lse.clone()
        g = torch.cuda.CUDAGraph()                   # the step as a graph
        with torch.cuda.graph(g):
            draft(q)
        out.zero_(), lse.zero_(), q.zero_()
        g.replay()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        assert L.dsv4sa_check_errors() == (0, 0)
        # ---- a path of each tree is accepted
        accepted = [int(rng.integers(0, len(p))) for p in parents]
        new_seq, new_pos, src = [], [], []
        for b, node in enumerate(accepted):
            for j in range(len(parents[b])):
                if masks[b][node] >> j & 1:
                    new_seq.append(b), new_pos.append(int(pos[start[b] + j])), src.append(int(start[b] + j))
        drafted = torch.empty(len(src), 512, dtype=torch.bfloat16, device="cuda")
        L.dsv4sa_cache_read(spec.win, spec.win_pt, i32(new_seq), args["entry"][torch.tensor(src, device="cuda")].contiguous(), drafted)
        spec.commit(new_seq, new_pos, rows, i32(src))
        ring = torch.empty_like(drafted)
        L.dsv4sa_cache_read(spec.win, spec.win_pt, i32(new_seq), i32(np.array(new_pos) % 128), ring)
        assert torch.equal(ring.view(torch.int16), drafted.view(torch.int16))     # the drafted rows' bits
        for b, p, t in zip(new_seq, new_pos, src):   # plain decoding of the same tokens
            o, l = plain.decode(b, p, x[t:t + 1], rows[t:t + 1])
            # each within its own tolerance of 64 bits; the plain one merges splits in BF16
            assert (o.float() - out[t].float()).abs().max() <= 2e-2, (step, b, t)
            assert (l - lse[t]).abs().max() <= 1e-3
        for b, node in enumerate(accepted):
            spec.ctx[b] += bin(masks[b][node]).count("1")
        plain.ctx = list(spec.ctx)
        ring_a, ring_b = (torch.empty(384, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        at = (i32(np.repeat(np.arange(3), 128)), i32(np.tile(np.arange(128), 3)))
        L.dsv4sa_cache_read(spec.win, spec.win_pt, *at, ring_a)
        L.dsv4sa_cache_read(plain.win, plain.win_pt, *at, ring_b)
        assert torch.equal(ring_a.view(torch.int16), ring_b.view(torch.int16))
    assert L.dsv4sa_check_errors() == (0, 0)
