"""Arrays of 32-bit values have to lie on 4 bytes: the C entry points refuse others before
anything is launched."""
import ctypes
import os

import pytest

from test_cache_norm_cpu import INVALID, OK, attn, cache, pool, ptr


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("field", ["attn_sink", "q_seq", "comp_pt", "idx_c", "win_pt", "idx_w", "win_pos", "lse", "rope_pos"])
def test_attention(L, field, off):
    pools = [(pool(L, k, 1), pool(L, k, 8)) for k in (L.POOL_KV_FP4, L.POOL_KV)]
    more = {"win_pos": dict(idx_w=None), "rope_pos": dict(rope_cs=ptr(950), rope_rows=8)}.get(field, {})
    for call in (L.lib().dsv4sa_sparse_attn_decode, L.lib().dsv4sa_sparse_attn_prefill):
        for comp, win in pools:
            a = attn(L, comp, win, **{**more, field: ptr(901, off)})
            assert call(ctypes.byref(a), None) == INVALID
            a.T = 0
            assert call(ctypes.byref(a), None) == OK              # nothing is read


@pytest.mark.parametrize("off", [1, 2])
def test_rows_and_pages(L, off):
    lib, big, bad = L.lib(), ptr(900), ptr(901, off)
    for kind, names in ((L.POOL_KV_FP4, ("cache_write", "cache_read")), (L.POOL_KV, ("cache_write", "cache_read")),
                        (L.POOL_IDXK_FP4, ("cache_write", "cache_write_rotated"))):
        p = ctypes.byref(pool(L, kind, 1))
        for name in names:
            call = getattr(lib, "dsv4sa_" + name)
            assert call(p, bad, 4, big, big, ptr(920), 3, None) == INVALID
            assert call(p, big, 4, bad, big, ptr(920), 3, None) == INVALID
            assert call(p, big, 4, big, bad, ptr(920), 3, None) == INVALID
    kv = pool(L, L.POOL_KV, 1)
    arr = (L.PoolDesc * 1)(kv)
    assert lib.dsv4sa_pages_copy(arr, 1, bad, big, 1, None) == INVALID and lib.dsv4sa_pages_copy(arr, 1, big, bad, 1, None) == INVALID
    c = ctypes.byref(cache(L, [kv]))
    assert lib.dsv4sa_cache_release(c, bad, 1, None) == INVALID
    for i in range(4):
        lists = [ptr(900), ptr(902), ptr(904), ptr(906)]
        lists[i] = bad
        assert lib.dsv4sa_cache_fork(c, *lists[:3], 1, lists[3], None) == INVALID
    assert lib.dsv4sa_cache_compact(c, c, bad, ptr(910), None) == INVALID
    assert lib.dsv4sa_cache_compact(c, c, ptr(910), bad, None) == INVALID
    crooked = cache(L, [kv])
    crooked.page_table = ptr(700, off)
    assert lib.dsv4sa_cache_release(ctypes.byref(crooked), big, 1, None) == INVALID
