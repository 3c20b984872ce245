"""The largest batches that the attention of drafted tokens takes (the call ends at the missing workspace)."""
import ctypes

import pytest

from test_cache_norm_cpu import UNSUPPORTED, pool
from test_drafts_cpu import L, WORKSPACE, tree_args  # noqa: F401


@pytest.mark.parametrize("n_seqs,nodes,heads,want", [
    (2 ** 24, 1, 1, WORKSPACE), (2 ** 24 + 1, 1, 1, UNSUPPORTED), (2 ** 31 - 1, 1, 1, UNSUPPORTED), (2 ** 24, 16, 64, WORKSPACE),
    (2 ** 24, 17, 64, UNSUPPORTED), (2 ** 21, 64, 128, WORKSPACE), (2 ** 21 + 1, 64, 128, UNSUPPORTED)])
def test_sequences_and_items(L, n_seqs, nodes, heads, want):
    kv, other = pool(L, L.POOL_KV, 1), pool(L, L.POOL_KV, 8)
    a = tree_args(L, kv, other, n_seqs=n_seqs, max_nodes=nodes, H=heads, ws=None)
    assert L.lib().dsv4sa_tree_attn(ctypes.byref(a), None) == want
