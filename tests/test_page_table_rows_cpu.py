"""Page tables of fewer rows than a call's sequences: refused before anything is launched."""
import ctypes
import os
import subprocess

import pytest

from test_abi_cpu import HEADER
from test_binding_devices_cpu import bf16, f32, i32, on
from test_cache_norm_cpu import INVALID, OK, pool, ptr
from test_drafts_cpu import L, WORKSPACE, append_args, gpu0, tree_args  # noqa: F401


def tree_call(L, B, comp_rows, win_rows, seq_row=None, n_max=9, window=128, draft=128):
    kv = L.PoolDesc()
    L.dsv4sa_tree_attn(on((3, 16, 512), bf16), on((16,), f32), on((B + 1,), i32), on((B,), i32), on((3,), i32), kv,
                       on((comp_rows, 4), i32), on((3,), i32), n_max, kv, on((win_rows, 4), i32), window, on((3, 16, 512), bf16), 0.04,
                       max_nodes=4, seq_row=seq_row, win_ring=128 if window else 0, draft_entry=draft)


def test_tree_binding_counts_table_rows(L, gpu0):
    tree_call(L, 3, 3, 4)
    tree_call(L, 3, 1, 3, n_max=0)                            # nothing is read from that table
    tree_call(L, 3, 3, 1, window=0, draft=-1)
    tree_call(L, 3, 2, 2, seq_row=on((3,), i32))              # rows by a list: checked on the device
    for bad in (dict(comp_rows=2, win_rows=3), dict(comp_rows=3, win_rows=2), dict(comp_rows=3, win_rows=2, window=0),
                dict(comp_rows=0, win_rows=3, seq_row=on((3,), i32))):
        with pytest.raises(ValueError, match="row"):
            tree_call(L, 3, **bad)
    assert L.lib.reached == ["dsv4sa_tree_attn"] * 4


def test_tree_call_counts_table_rows(L):
    kv, other = pool(L, L.POOL_KV, 1), pool(L, L.POOL_KV, 8)

    def st(**kw):
        return L.lib().dsv4sa_tree_attn(ctypes.byref(tree_args(L, kv, other, ws=None, **kw)), None)
    assert st(n_seqs=2, comp_pt_rows=2, win_pt_rows=2) == WORKSPACE        # accepted up to there
    assert st(n_seqs=2) == WORKSPACE                                       # not told
    assert st(n_seqs=2, comp_pt_rows=1, win_pt_rows=1, seq_row=ptr(1)) == WORKSPACE
    assert st(n_seqs=2, comp_pt_rows=1, n_max=0, comp_pt=None) == WORKSPACE
    for bad in (dict(comp_pt_rows=1), dict(win_pt_rows=1), dict(comp_pt_rows=-1), dict(win_pt_rows=-1), dict(win_pt_rows=1, window=0)):
        assert st(n_seqs=2, **bad) == INVALID, bad


def test_append_counts_table_rows(L, gpu0):
    rows, seq = on((5, 512), bf16), on((5,), i32)
    L.dsv4sa_cache_append(L.PoolDesc(), on((2, 4), i32), seq, seq, rows)
    L.dsv4sa_cache_append(L.PoolDesc(), on((0, 4), i32), seq[:0], seq[:0], rows[:0])
    L.dsv4sa_cache_append(L.PoolDesc(), on((4,), i32), seq, seq, rows)           # a table of one row
    for table in ((0, 4), (2, 0, 4)):
        with pytest.raises(ValueError, match="row"):
            L.dsv4sa_cache_append(L.PoolDesc(), on(table, i32), seq, seq, rows)
    assert L.lib.reached == ["dsv4sa_cache_append"] * 3


def test_append_call_refuses_negative_table_rows(L):
    p = pool(L, L.POOL_KV, 1)
    assert L.lib().dsv4sa_cache_append(ctypes.byref(append_args(L, p, n=0, pt_rows=3)), None) == OK
    assert L.lib().dsv4sa_cache_append(ctypes.byref(append_args(L, p, pt_rows=-1)), None) == INVALID


@pytest.mark.parametrize("struct,name,fields", [("TreeArgs", "dsv4sa_tree_args", ["seq_row", "ws_bytes", "comp_pt_rows", "win_pt_rows"]),
                                                ("AppendArgs", "dsv4sa_append_args", ["row_entry", "norm_w", "eps", "pt_rows"])])
def test_struct_is_the_headers(L, tmp_path, struct, name, fields):
    """The binding's structure has the header's size and offsets."""
    src, exe = tmp_path / "s.c", tmp_path / "s"
    offsets = "".join(f', (int)offsetof({name}, {f})' for f in fields)
    src.write_text(f'#include <stdio.h>\n#include "dsv4sa.h"\n'
                   f'int main(void) {{ printf("%d{" %d" * len(fields)}\\n", (int)sizeof({name}){offsets}); return 0; }}\n')
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), "-I", "/usr/local/cuda/include", "-o", str(exe), str(src)], check=True)
    args = getattr(L, struct)
    want = [ctypes.sizeof(args)] + [getattr(args, f).offset for f in fields]
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want
