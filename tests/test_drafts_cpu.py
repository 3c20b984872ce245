"""Rotary positions, appended rows and drafted tokens on a host without a GPU: what the library
and its binding refuse before anything is launched."""
import ctypes
import math
import os

import pytest
import torch

from test_binding_devices_cpu import bf16, f32, i32, on, u8
from test_cache_norm_cpu import INVALID, OK, UNSUPPORTED, pool, ptr

WORKSPACE = 3


class Lib:
    """A library whose entry points only count that they were reached."""

    def __init__(self):
        self.reached = []

    def __call__(self):
        return self

    def __getattr__(self, fn):
        return lambda *a: self.reached.append(fn) or 0


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.fixture
def gpu0(L, monkeypatch):
    """The binding as on a host whose current device is cuda:0, the library never reached."""
    monkeypatch.setattr(L, "_here", lambda: 0)
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_stream", lambda s, here=None: 0)
    monkeypatch.setattr(L, "lib", Lib())


def test_table(L):
    def st(cs=ptr(900), rows=4, pairs=32, first=0, base=1e4, factor=1.0, length=0, fast=32.0, slow=1.0):
        return L.lib().dsv4sa_rope_table(cs, rows, pairs, first, base, factor, length, fast, slow, None)
    assert st(rows=0, cs=None) == OK
    for bad in (dict(cs=None), dict(cs=ptr(900, 4)), dict(rows=-1), dict(pairs=0), dict(first=-1), dict(first=2 ** 63 - 2), dict(base=1.0),
                dict(base=math.nan), dict(base=math.inf), dict(base=-2.0), dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf),
                dict(length=-1), dict(length=100, slow=0.0), dict(length=100, fast=1.0, slow=2.0), dict(length=100, fast=math.nan)):
        assert st(**bad) == INVALID, bad
    assert st(pairs=257) == UNSUPPORTED


def test_table_binding(L, gpu0):
    with pytest.raises(ValueError):
        L.dsv4sa_rope_table(on((4, 32), f32))


def rope_args(L, **kw):
    a = L.RopeArgs(ptr(900), 8 * 512, 512, ptr(910), 8 * 512, 512, 3, 8, 512, 448, 64, 0, 0, 100, ptr(920), ptr(930), 1, 1e-6, ptr(940))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_rope(L):
    def st(**kw):
        return L.lib().dsv4sa_rope(ctypes.byref(rope_args(L, **kw)), None)
    assert L.lib().dsv4sa_rope(None, None) == INVALID
    assert st(T=0) == OK and st(T=0, x=None, pos=None) == OK
    for bad in (dict(x=None), dict(out=None), dict(x=ptr(900, 8)), dict(out=ptr(910, 2)), dict(pos=None), dict(pos=ptr(930, 2)),
                dict(rope_cs=None), dict(rope_cs=ptr(920, 8)), dict(rope_rows=0), dict(norm_w=ptr(940, 4)), dict(T=-1), dict(H=0),
                dict(dim=0), dict(dim=508), dict(rope_dim=8), dict(rope_dim=24), dict(rope_dim=0), dict(rope_off=456), dict(rope_off=-8),
                dict(rope_off=444), dict(layout=2), dict(inverse=2), dict(norm=3), dict(eps=-1.0), dict(eps=math.nan),
                dict(x_tok_stride=-8), dict(x_head_stride=516), dict(out_head_stride=504), dict(out_tok_stride=7 * 512),
                dict(out_tok_stride=0), dict(out_head_stride=0), dict(x_tok_stride=2 ** 41)):
        assert st(**bad) == INVALID, bad
    for big in (dict(dim=1032, out_head_stride=1032, out_tok_stride=9000), dict(rope_dim=528, dim=1024, rope_off=0, out_head_stride=1024,
                                                                               out_tok_stride=9000), dict(T=2 ** 28, H=8)):
        assert st(**big) == UNSUPPORTED, big
    # out within x, or over the table, positions or weights
    span = 3 * 8 * 512 * 2
    assert st(out=ptr(900, 16)) == INVALID and st(out=ptr(900, span - 16)) == INVALID
    assert st(out=ptr(900), out_tok_stride=16 * 512) == INVALID          # x's start, other strides
    assert st(rope_cs=ptr(910, 32)) == INVALID and st(pos=ptr(910, 64)) == INVALID and st(norm_w=ptr(910, span - 16)) == INVALID


def test_rope_binding(L, gpu0):
    x, cs, pos = on((4, 3, 128), bf16), on((10, 32, 2), f32), on((4,), i32)
    for call in (lambda: L.dsv4sa_rope(on((4, 128), bf16), cs, pos), lambda: L.dsv4sa_rope(x, on((10, 32), f32), pos),
                 lambda: L.dsv4sa_rope(x, cs, on((3,), i32)), lambda: L.dsv4sa_rope(x, cs, pos, out=on((4, 3, 120), bf16)),
                 lambda: L.dsv4sa_rope(x, cs, pos, norm_w=on((128,), f32)),
                 lambda: L.dsv4sa_rope(x, cs, pos, eps=1e-6, norm_w=on((64,), f32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        L.dsv4sa_rope(torch.zeros(4, 3, 128, dtype=torch.bfloat16), cs, pos)


def append_args(L, p, **kw):
    a = L.AppendArgs(ctypes.pointer(p), ptr(900), 4, 0, ptr(910), ptr(920), None, None, ptr(930), 512, 8, 8, ptr(940), 100, 1, ptr(950), 1e-6, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_append(L):
    for kind in (L.POOL_KV, L.POOL_KV_FP4):
        p = pool(L, kind, 1)

        def st(**kw):
            return L.lib().dsv4sa_cache_append(ctypes.byref(append_args(L, p, **kw)), None)
        assert st(n=0) == OK and st(n=0, rows=None) == OK
        for bad in (dict(n=-1), dict(n_src=-1), dict(n_src=7), dict(n_src=0, src_row=ptr(960)), dict(pt_stride=0), dict(ring=-1),
                    dict(norm=2), dict(eps=-1.0), dict(eps=math.nan), dict(row_stride=504), dict(row_stride=516), dict(rows=None),
                    dict(rows=ptr(930, 8)), dict(page_table=None), dict(page_table=ptr(900, 2)), dict(row_seq=None), dict(row_seq=ptr(910, 1)),
                    dict(row_pos=ptr(920, 2)), dict(row_entry=ptr(960, 2)), dict(src_row=ptr(960, 3)), dict(norm_w=ptr(950, 4)),
                    dict(rope_cs=ptr(940, 8)), dict(rope_rows=0), dict(row_pos=None), dict(row_pos=None, row_entry=ptr(960)),
                    dict(row_pos=None, rope_cs=None), dict(rows=ptr(1, 4096)), dict(pool=None)):
            assert st(**bad) == INVALID, bad
    for kind in (L.POOL_IDXK, L.POOL_IDXK_FP4):
        p = pool(L, kind, 1)
        assert L.lib().dsv4sa_cache_append(ctypes.byref(append_args(L, p)), None) == INVALID
    assert L.lib().dsv4sa_cache_append(None, None) == INVALID


def test_append_binding(L, gpu0):
    p = L.PoolDesc()
    pt, seq, rows = on((2, 4), i32), on((5,), i32), on((5, 512), bf16)
    for call in (lambda: L.dsv4sa_cache_append(p, pt, seq, seq, on((4, 512), bf16)), lambda: L.dsv4sa_cache_append(p, pt, seq, seq, on((5, 256), bf16)),
                 lambda: L.dsv4sa_cache_append(p, pt, seq, on((4,), i32), rows), lambda: L.dsv4sa_cache_append(p, pt, seq, seq, rows, row_entry=on((4,), i32)),
                 lambda: L.dsv4sa_cache_append(p, pt, seq, seq, rows, src_row=on((4,), i32)),
                 lambda: L.dsv4sa_cache_append(p, pt, seq, seq, rows, on((9, 16, 2), f32)),
                 lambda: L.dsv4sa_cache_append(p, pt, seq, seq, rows, norm_w=on((512,), f32)),
                 lambda: L.dsv4sa_cache_append(p, pt, seq, seq, rows, eps=1e-6, norm_w=on((64,), f32))):
        with pytest.raises(ValueError):
            call()


def tree_args(L, comp, win, **kw):
    a = L.TreeArgs()
    a.T, a.H, a.softmax_scale, a.n_seqs, a.n_max, a.max_nodes, a.window, a.win_ring, a.draft_entry = 6, 64, 0.04, 2, 200, 4, 128, 128, 128
    for i, f in enumerate(("q", "attn_sink", "node_start", "ctx", "pos", "n_vis", "comp_pt", "win_pt", "out", "ws")):
        setattr(a, f, ptr(700 + 60 * i))
    a.comp, a.win = ctypes.pointer(comp) if comp else None, ctypes.pointer(win) if win else None
    a.comp_pt_stride = a.win_pt_stride = 4
    a.ws_bytes = 64 * MB_WS
    for k, v in kw.items():
        setattr(a, k, v)
    return a


MB_WS = 1 << 20


def test_tree_attention(L):
    kv, other = pool(L, L.POOL_KV, 1), pool(L, L.POOL_KV, 8)
    f4, keys = pool(L, L.POOL_KV_FP4, 16), pool(L, L.POOL_IDXK, 24)

    def st(comp=kv, win=other, **kw):
        return L.lib().dsv4sa_tree_attn(ctypes.byref(tree_args(L, comp, win, **kw)), None)
    assert L.lib().dsv4sa_tree_attn(None, None) == INVALID
    for nothing in (dict(T=0), dict(n_seqs=0), dict(max_nodes=0)):
        assert st(q=None, **nothing) == OK
    for bad in (dict(q=None), dict(q=ptr(700, 8)), dict(out=ptr(701, 2)), dict(out=None), dict(attn_sink=None), dict(attn_sink=ptr(1, 2)),
                dict(node_start=None), dict(node_start=ptr(1, 1)), dict(ctx=None), dict(ctx=ptr(1, 2)), dict(pos=None), dict(pos=ptr(1, 3)),
                dict(n_vis=None), dict(n_vis=ptr(1, 2)), dict(anc=ptr(1, 4)), dict(seq_row=ptr(1, 2)), dict(lse=ptr(1, 2)),
                dict(comp_pt=None), dict(win_pt=None), dict(comp_pt=ptr(1, 2)), dict(win_pt=ptr(1, 2)), dict(comp=None), dict(win=None),
                dict(comp=keys), dict(win=keys), dict(n_max=257), dict(comp_pt_stride=0), dict(win_pt_stride=0), dict(win_ring=257),
                dict(T=-1), dict(n_seqs=-1), dict(max_nodes=-1), dict(n_max=-1), dict(window=-1), dict(win_ring=-1), dict(draft_entry=-2),
                dict(rope_cs=ptr(1)), dict(rope_cs=ptr(1), rope_pos=ptr(2)), dict(rope_cs=ptr(1, 8), rope_pos=ptr(2), rope_rows=9),
                dict(out=ptr(700, 1024))):
        assert st(**bad) == INVALID, bad
    for big in (dict(H=0), dict(H=129), dict(max_nodes=65), dict(n_max=2 ** 29 + 1, comp_pt_stride=2 ** 24), dict(window=65537),
                dict(draft_entry=2 ** 30 + 1), dict(T=2 ** 25), dict(n_seqs=2 ** 30), dict(comp=f4), dict(win=f4)):
        assert st(**big) == UNSUPPORTED, big
    assert st(ws=None) == WORKSPACE and st(ws=ptr(1, 8)) == WORKSPACE
    need = L.dsv4sa_tree_attn_workspace_size(2, 4, 64, 200, 128)
    assert st(ws_bytes=need - 1) == WORKSPACE
    # pools that nothing would be read from need not be there
    assert st(comp=None, comp_pt=None, n_max=0, ws=None) == WORKSPACE
    assert st(win=None, win_pt=None, window=0, draft_entry=-1, ws=None) == WORKSPACE


def test_workspace_size(L):
    size = L.dsv4sa_tree_attn_workspace_size
    assert size(0, 1, 1, 1, 1) == size(1, 0, 1, 1, 1) == size(1, 65, 1, 1, 1) == size(1, 1, 129, 1, 1) == size(1, 1, 1, -1, 1) == 0
    assert 0 < size(1, 1, 16, 0, 0) < size(1, 1, 16, 8192, 128) <= 42.2e6 and size(4096, 64, 128, 2 ** 29, 65536) <= 42.2e6


def test_window_lists(L):
    def st(start=ptr(900), ctx=ptr(910), pos=ptr(920), anc=None, n_seqs=2, T=6, nodes=4, window=128, ring=128, draft=128, idx=ptr(930), stride=132):
        return L.lib().dsv4sa_tree_window_indices(start, ctx, pos, anc, n_seqs, T, nodes, window, ring, draft, idx, stride, None)
    for nothing in (dict(n_seqs=0), dict(T=0), dict(nodes=0)):
        assert st(idx=None, **nothing) == OK
    for bad in (dict(start=None), dict(start=ptr(1, 2)), dict(ctx=None), dict(ctx=ptr(1, 1)), dict(pos=None), dict(pos=ptr(1, 2)),
                dict(anc=ptr(1, 4)), dict(idx=None), dict(idx=ptr(1, 2)), dict(n_seqs=-1), dict(T=-1), dict(nodes=-1), dict(window=-1),
                dict(ring=-1), dict(draft=-2), dict(stride=131)):
        assert st(**bad) == INVALID, bad
    for big in (dict(nodes=65, stride=300), dict(window=65537, stride=70000), dict(draft=2 ** 30 + 1)):
        assert st(**big) == UNSUPPORTED, big


def test_tree_binding(L, gpu0):
    kv = L.PoolDesc()
    t = dict(q=on((3, 16, 512), bf16), sink=on((16,), f32), start=on((3,), i32), ctx=on((2,), i32), pos=on((3,), i32), pt=on((2, 4), i32),
             n_vis=on((3,), i32), out=on((3, 16, 512), bf16), anc=on((3,), torch.int64))

    def call(**kw):
        a = {**t, **{k: v for k, v in kw.items() if k in t}}
        more = {k: v for k, v in kw.items() if k not in t}
        L.dsv4sa_tree_attn(a["q"], a["sink"], a["start"], a["ctx"], a["pos"], kv, a["pt"], a["n_vis"], 9, kv, a["pt"], 128, a["out"], 0.04,
                           max_nodes=4, anc=a["anc"], win_ring=128, draft_entry=128, **more)
    for bad in (dict(q=on((3, 16, 256), bf16)), dict(out=on((2, 16, 512), bf16)), dict(sink=on((8,), f32)), dict(ctx=on((1,), i32)),
                dict(pos=on((2,), i32)), dict(n_vis=on((2,), i32)), dict(anc=on((2,), torch.int64)), dict(lse=on((3, 8), f32)),
                dict(seq_row=on((1,), i32)), dict(rope_cs=on((9, 16, 2), f32), rope_pos=on((3,), i32)),
                dict(rope_cs=on((9, 32, 2), f32), rope_pos=on((2,), i32))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(anc=on((3,), i32)), dict(q=on((3, 16, 512), f32)), dict(ws=on((64,), f32))):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(ValueError):
        L.dsv4sa_tree_window_indices(t["start"], t["ctx"], t["pos"], 128, 128, 128, 4, on((400,), i32))


def device_calls(L):
    """name -> (tensors by name, pools by name, the call)."""
    def tree(t, p):
        L.dsv4sa_tree_attn(t["q"], t["sink"], t["start"], t["ctx"], t["pos"], p["comp"], t["comp_pt"], t["n_vis"], 9, p["win"], t["win_pt"],
                           128, t["out"], 0.04, max_nodes=4, anc=t["anc"], seq_row=t["seq_row"], lse=t["lse"], ws=t["ws"],
                           rope_cs=t["rope_cs"], rope_pos=t["pos"])
    nodes = dict(start=((3,), i32), ctx=((2,), i32), pos=((3,), i32), anc=((3,), torch.int64))
    return {
        "dsv4sa_rope_table": (dict(cs=((4, 32, 2), f32)), [], lambda t, p: L.dsv4sa_rope_table(t["cs"])),
        "dsv4sa_rope": (dict(x=((3, 2, 128), bf16), out=((3, 2, 128), bf16), cs=((4, 32, 2), f32), pos=((3,), i32), w=((128,), f32)), [],
                        lambda t, p: L.dsv4sa_rope(t["x"], t["cs"], t["pos"], out=t["out"], eps=1e-6, norm_w=t["w"])),
        "dsv4sa_cache_append": (dict(pt=((2, 4), i32), seq=((3,), i32), pos=((3,), i32), ent=((3,), i32), src=((3,), i32), rows=((3, 512), bf16),
                                     cs=((4, 32, 2), f32), w=((512,), f32)), ["pool"],
                                lambda t, p: L.dsv4sa_cache_append(p["pool"], t["pt"], t["seq"], t["pos"], t["rows"], t["cs"], row_entry=t["ent"],
                                                                   src_row=t["src"], eps=1e-6, norm_w=t["w"])),
        "dsv4sa_tree_attn": (dict(q=((3, 16, 512), bf16), out=((3, 16, 512), bf16), sink=((16,), f32), comp_pt=((2, 4), i32), win_pt=((2, 4), i32),
                                  n_vis=((3,), i32), seq_row=((2,), i32), lse=((3, 16), f32), ws=((64,), u8), rope_cs=((4, 32, 2), f32), **nodes),
                             ["comp", "win"], tree),
        "dsv4sa_tree_window_indices": (dict(idx=((3, 132), i32), **nodes), [],
                                       lambda t, p: L.dsv4sa_tree_window_indices(t["start"], t["ctx"], t["pos"], 128, 128, 128, 4, t["idx"],
                                                                                 anc=t["anc"])),
    }


@pytest.mark.parametrize("name", ["dsv4sa_rope_table", "dsv4sa_rope", "dsv4sa_cache_append", "dsv4sa_tree_attn", "dsv4sa_tree_window_indices"])
def test_every_tensor_has_to_be_on_the_current_device(L, name, monkeypatch):
    tensors, pools, call = device_calls(L)[name]
    fake = Lib()
    reached = fake.reached
    monkeypatch.setattr(L, "_here", lambda: 0)
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_stream", lambda s, here=None: 0)
    descs = {n: pool(L, L.POOL_KV, 1 + 8 * i) for i, n in enumerate(pools)}
    monkeypatch.setattr(L, "lib", fake)
    call({n: on(s, d) for n, (s, d) in tensors.items()}, descs)
    assert reached == [name]
    for wrong in tensors:
        with pytest.raises(ValueError, match="current device"):
            call({n: on(s, d, 1 if n == wrong else 0) for n, (s, d) in tensors.items()}, descs)
    for wrong in pools:
        descs[wrong].device = 1
        with pytest.raises(ValueError, match="current device"):
            call({n: on(s, d) for n, (s, d) in tensors.items()}, descs)
        descs[wrong].device = None
    assert reached == [name]
