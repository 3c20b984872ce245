"""FP4 KV cache, pages and norm on a host without a GPU: the page's layout, and what the
library and its binding refuse before anything is launched."""
import ctypes
import os

import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def ptr(mb, extra=0):
    """A made-up device address: the calls here end before anything reads it."""
    return ctypes.c_void_p(mb * MB + extra)


def pool(L, kind, mb, pages=4):
    return L.dsv4sa_pool_desc_init(kind, mb * MB, pages)


def test_status_of_no_pages(L):
    assert L.lib().dsv4sa_status_string(7).decode() == L.STATUS[7]


def test_kv_fp4_layout(L):
    assert L.dsv4sa_pool_bytes(L.POOL_KV_FP4, 3) == 3 * 23552
    d = pool(L, L.POOL_KV_FP4, 1, 10)
    assert (d.page_stride, d.nope_off, d.rope_off, d.scale_off) == (23552, 0, 14336, 22528)
    assert (d.nope_row, d.rope_row, d.scale_row, d.n_scales, d.scale_group) == (224, 128, 16, 14, 32)
    assert d.rope_off == 64 * d.nope_row and d.scale_off == d.rope_off + 64 * d.rope_row
    assert d.page_stride == d.scale_off + 64 * d.scale_row and d.page_stride % 1024 == 0
    for v in (d.nope_row, d.rope_row, d.scale_row, d.rope_off, d.scale_off):
        assert v % 16 == 0
    with pytest.raises(L.DSV4SAError):
        L.dsv4sa_pool_desc_init(L.POOL_KV_FP4, MB + 512, 10)


def attn(L, comp, win, kc=512, kw=128, **kw_args):
    a = L.AttnArgs()
    a.T, a.H, a.softmax_scale = 2, 64, 0.04
    for f in ("q", "attn_sink", "q_seq", "out", "comp_pt", "win_pt", "idx_c", "idx_w"):
        setattr(a, f, ptr(900))
    a.comp, a.win = ctypes.pointer(comp) if comp else None, ctypes.pointer(win) if win else None
    a.kc = a.idx_c_stride = kc
    a.kw = a.idx_w_stride = kw
    a.comp_pt_stride = a.win_pt_stride = 64
    for k, v in kw_args.items():
        setattr(a, k, v)
    return a


def test_attention_refusals(L):
    lib = L.lib()
    kv, f4, f4b = pool(L, L.POOL_KV, 1), pool(L, L.POOL_KV_FP4, 8), pool(L, L.POOL_KV_FP4, 16)
    keys = pool(L, L.POOL_IDXK_FP4, 24)
    broken = pool(L, L.POOL_KV_FP4, 32)
    broken.scale_row = 14
    for call in (lib.dsv4sa_sparse_attn_decode, lib.dsv4sa_sparse_attn_prefill):
        def st(*args, **kw):
            return call(ctypes.byref(attn(L, *args, **kw)), None)
        assert st(kv, f4) == UNSUPPORTED and st(f4, kv) == UNSUPPORTED           # one of each
        assert st(f4, keys) == INVALID and st(keys, f4) == INVALID and st(keys, keys) == INVALID
        assert st(f4, broken) == INVALID and st(broken, f4) == INVALID
        assert st(f4, f4b, idx_c_stride=511) == INVALID and st(f4, f4b, idx_w_stride=127) == INVALID
        assert st(f4, f4b, comp_pt_stride=0) == INVALID and st(f4, f4b, win_pt=None) == INVALID
        assert st(f4, f4b, q=ptr(900, 8)) == INVALID and st(f4, f4b, out=ptr(900, 8)) == INVALID
        assert st(f4, f4b, H=0) == UNSUPPORTED and st(f4, f4b, H=129) == UNSUPPORTED
        assert st(f4, f4b, kc=-1) == INVALID and st(f4, f4b, T=-1) == INVALID
        assert st(f4, f4b, kc=1 << 30, idx_c_stride=1 << 30, kw=1, idx_w_stride=1) == UNSUPPORTED
        assert st(None, f4) == INVALID and st(f4, None) == INVALID
        assert st(f4, f4b, rope_cs=ptr(900)) == INVALID                             # a table without positions
        assert st(f4, f4b, T=0) == OK


def test_cache_rows_refusals(L):
    lib, p, big = L.lib(), pool(L, L.POOL_KV_FP4, 1), ptr(900)
    bad = pool(L, L.POOL_KV_FP4, 1)
    bad.rope_off += 16
    for name in ("dsv4sa_cache_write", "dsv4sa_cache_read"):
        call = getattr(lib, name)
        assert call(ctypes.byref(p), big, 4, big, big, big, 0, None) == OK
        assert call(ctypes.byref(p), big, 4, big, big, big, -1, None) == INVALID
        assert call(ctypes.byref(p), big, 0, big, big, big, 3, None) == INVALID
        assert call(ctypes.byref(bad), big, 4, big, big, big, 3, None) == INVALID
        assert call(ctypes.byref(p), None, 4, big, big, big, 3, None) == INVALID
        assert call(ctypes.byref(p), big, 4, None, big, big, 3, None) == INVALID
        assert call(ctypes.byref(p), big, 4, big, None, big, 3, None) == INVALID
        assert call(ctypes.byref(p), big, 4, big, big, ptr(900, 2), 3, None) == INVALID
        assert call(None, big, 4, big, big, big, 3, None) == INVALID
    assert lib.dsv4sa_cache_write_rotated(ctypes.byref(p), big, 4, big, big, big, 3, None) == INVALID
    for kind in (L.POOL_IDXK, L.POOL_IDXK_FP4):                 # keys are not read back
        assert lib.dsv4sa_cache_read(ctypes.byref(pool(L, kind, 1)), big, 4, big, big, big, 3, None) == INVALID
    end = MB + 4 * 23552                                         # rows inside the pool, or reaching into it
    for at in (MB, MB + 1024, end - 16, MB - 3 * 1024 + 16):
        assert lib.dsv4sa_cache_read(ctypes.byref(p), big, 4, big, big, ctypes.c_void_p(at), 3, None) == INVALID


def cache(L, pools, rows=8, stride=16, table=700, use=710, use_extra=0):
    arr = (L.PoolDesc * len(pools))(*pools)
    c = L.CacheDesc()
    c._keep = arr
    c.pools, c.n_pools, c.rows, c.pt_stride = ctypes.cast(arr, ctypes.POINTER(L.PoolDesc)), len(pools), rows, stride
    c.page_table, c.use = ptr(table), ptr(use, use_extra)
    return c


def test_pages_refusals(L):
    lib, big = L.lib(), ptr(900)
    kv, f4, keys = pool(L, L.POOL_KV, 1), pool(L, L.POOL_KV_FP4, 8), pool(L, L.POOL_IDXK_FP4, 16)

    def copy(pools, n=1, src=big, dst=big):
        arr = (L.PoolDesc * max(1, len(pools)))(*pools)
        return lib.dsv4sa_pages_copy(arr, len(pools), src, dst, n, None)
    assert copy([kv, f4, keys], 0) == OK
    assert copy([]) == INVALID and copy([kv] * 5) == INVALID and copy([kv], -1) == INVALID
    assert copy([kv], src=None) == INVALID and copy([kv], dst=None) == INVALID
    assert copy([kv], (1 << 28) + 1) == UNSUPPORTED
    assert copy([kv, pool(L, L.POOL_KV_FP4, 8, 5)]) == INVALID                  # not the same pages
    assert copy([kv, kv]) == INVALID                                            # the same memory twice
    broken = pool(L, L.POOL_KV, 1)
    broken.page_stride *= 2
    assert copy([broken]) == INVALID

    bad = [cache(L, [kv], rows=0), cache(L, [kv], stride=0), cache(L, [kv], use_extra=4), cache(L, [kv, kv]), cache(L, [broken])]
    for field in ("page_table", "use", "pools"):
        c = cache(L, [kv])
        setattr(c, field, None)
        bad.append(c)
    good = cache(L, [kv, keys])
    for c in bad:
        r = ctypes.byref(c)
        assert lib.dsv4sa_cache_release(r, big, 1, None) == INVALID
        assert lib.dsv4sa_cache_fork(r, big, big, big, 1, ptr(901), None) == INVALID
        assert lib.dsv4sa_cache_compact(r, r, big, ptr(901), None) == INVALID
        assert lib.dsv4sa_cache_compact(ctypes.byref(good), r, big, ptr(901), None) == INVALID
    r = ctypes.byref(good)
    assert lib.dsv4sa_cache_release(r, big, 0, None) == OK and lib.dsv4sa_cache_release(r, big, -1, None) == INVALID
    assert lib.dsv4sa_cache_release(r, None, 1, None) == INVALID
    assert lib.dsv4sa_cache_fork(r, big, big, big, 0, ptr(901), None) == OK
    assert lib.dsv4sa_cache_fork(r, big, big, big, -1, ptr(901), None) == INVALID
    assert lib.dsv4sa_cache_fork(r, big, big, big, (1 << 28) + 1, ptr(901), None) == UNSUPPORTED
    assert lib.dsv4sa_cache_fork(r, big, big, big, 1, None, None) == INVALID
    for where in (big, ptr(700, 8), ptr(710, 4), ptr(1, 64)):                   # new_page over an input, the table, the counts, a pool
        assert lib.dsv4sa_cache_fork(r, big, big, big, 1, where, None) == INVALID


def test_compact_refusals(L):
    lib = L.lib()
    kv, keys = pool(L, L.POOL_KV, 1), pool(L, L.POOL_IDXK_FP4, 16)
    src = cache(L, [kv, keys])

    def st(dst, new_id=ptr(900), n_used=ptr(901)):
        return lib.dsv4sa_cache_compact(ctypes.byref(src), ctypes.byref(dst), new_id, n_used, None)
    kv2, keys2 = pool(L, L.POOL_KV, 101), pool(L, L.POOL_IDXK_FP4, 116)
    apart = dict(table=800, use=810)
    assert st(cache(L, [kv2], **apart)) == INVALID                              # another number of pools, rows, entries
    assert st(cache(L, [kv2, keys2], rows=9, **apart)) == INVALID
    assert st(cache(L, [kv2, keys2], stride=15, **apart)) == INVALID
    assert st(cache(L, [keys2, kv2], **apart)) == INVALID                       # other kinds
    assert st(cache(L, [kv, keys2], **apart)) == INVALID                        # one pool shared
    assert st(cache(L, [kv, keys], **apart)) == INVALID                         # the pools in place, the table not
    assert st(cache(L, [kv2, keys2], table=700, use=810)) == INVALID            # the table shared
    assert st(cache(L, [kv2, keys2], table=800, use=710)) == INVALID            # the counts shared
    assert st(cache(L, [kv2, keys2], table=710, use=810)) == INVALID            # a table over the counts
    assert st(cache(L, [pool(L, L.POOL_KV, 16), keys2], **apart)) == INVALID    # a pool over another one's memory
    good = cache(L, [kv2, keys2], **apart)
    for where in (None, ptr(700), ptr(710), ptr(800), ptr(810), ptr(1), ptr(101), ptr(116, 64)):
        assert st(good, new_id=where) == INVALID and st(good, n_used=where) == INVALID
    assert st(good, new_id=ptr(900), n_used=ptr(900, 8)) == INVALID


def test_norm_refusals(L):
    lib = L.lib()
    x, r, w, ro, y, c, s = (ptr(m) for m in (100, 200, 300, 400, 500, 600, 700))

    def st(x=x, xs=256, res=None, rs=256, w=w, eps=1e-6, n=4, dim=256, group=128, ro=None, y=None, c=c, s=s):
        return lib.dsv4sa_rmsnorm_quant(x, xs, res, rs, w, eps, n, dim, group, ro, y, c, s, None)
    assert st(n=0) == OK and st(n=-1) == INVALID
    assert st(dim=0) == INVALID and st(dim=252) == INVALID and st(dim=16392, xs=16392) == UNSUPPORTED
    assert st(group=32) == UNSUPPORTED and st(group=0) == UNSUPPORTED
    assert st(dim=192, group=128) == INVALID                                    # codes need whole groups
    assert st(xs=248) == INVALID and st(xs=260) == INVALID                      # rows overlapping, rows off 16 bytes
    assert st(res=r, rs=248) == INVALID and st(res=r, rs=257) == INVALID
    assert st(eps=-1.0) == INVALID and st(eps=float("nan")) == INVALID
    assert st(c=None) == INVALID and st(s=None) == INVALID                      # codes and scales go together
    assert st(c=None, s=None) == INVALID                                        # no output at all
    assert st(x=None) == INVALID and st(w=None) == INVALID
    for name, at in (("x", 100), ("w", 300), ("ro", 400), ("y", 500), ("c", 600)):
        assert st(**{name: ptr(at, 8)}) == INVALID
    assert st(res=ptr(200, 8)) == INVALID and st(s=ptr(700, 2)) == INVALID
    # outputs over inputs, or over one another
    for name in ("y", "c", "s"):
        assert st(**{name: x}) == INVALID and st(res=r, **{name: r}) == INVALID and st(**{name: w}) == INVALID
        assert st(**{name: ptr(100, 4 * 512 - 16)}) == INVALID
    assert st(ro=x, xs=512) == INVALID and st(res=r, rs=264, ro=r) == INVALID   # in place, but with gaps
    assert st(ro=ptr(100, 16)) == INVALID and st(ro=w) == INVALID
    assert st(ro=y, y=y) == INVALID and st(y=c) == INVALID and st(y=ptr(700)) == INVALID


def test_binding_refuses(L):
    """Host tensors, wrong types and wrong shapes: errors of the binding."""
    f4 = pool(L, L.POOL_KV_FP4, 1)
    i32 = torch.zeros(4, dtype=torch.int32)
    rows = torch.zeros(4, 512, dtype=torch.bfloat16)
    for call in (L.dsv4sa_cache_write, L.dsv4sa_cache_read):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(f4, i32[None], i32, i32, rows)
        with pytest.raises(ValueError, match="512"):
            call(f4, i32[None], i32, i32, rows[:, :128])
    with pytest.raises(ValueError):
        L.dsv4sa_cache_read(f4, i32[None], i32[:3], i32, rows)
    with pytest.raises(ValueError):
        L.dsv4sa_cache_read(f4, i32[None], i32, i32, rows[:3])
    with pytest.raises(ValueError, match="1 to 4"):
        L.dsv4sa_pages_copy([], i32, i32)
    with pytest.raises(ValueError, match="1 to 4"):
        L.dsv4sa_pages_copy([f4] * 5, i32, i32)
    with pytest.raises(ValueError, match="length"):
        L.dsv4sa_pages_copy([f4], i32, i32[:3])
    with pytest.raises(ValueError, match="CUDA tensor"):
        L.dsv4sa_pages_copy([f4], i32, i32)
    with pytest.raises(ValueError, match="pt_stride"):
        L.page_cache([f4], i32, i32)
    with pytest.raises(ValueError, match="one count per page"):
        L.page_cache([f4], i32[None], i32[:3])
    with pytest.raises(ValueError, match="CUDA tensor"):
        L.page_cache([f4], i32[None], i32)
    c = cache(L, [f4])
    with pytest.raises(ValueError, match="length"):
        L.dsv4sa_cache_fork(c, i32, i32, i32[:3], i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        L.dsv4sa_cache_fork(c, i32, i32, i32, i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        L.dsv4sa_cache_release(c, i32)
    with pytest.raises(ValueError, match="one entry per page"):
        L.dsv4sa_cache_compact(c, c, i32[:3], i32[:1])
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    with pytest.raises(ValueError, match="CUDA tensor"):
        L.dsv4sa_rmsnorm_quant(x, w, y=x)
    with pytest.raises(ValueError, match="norm_w"):
        L.dsv4sa_rmsnorm_quant(x, w[:128], y=x)


def test_packed_fp4_pool_reads_back_on_the_host(L):
    """pack_kv_pool_fp4 places logical arrays by the page's layout."""
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (2, 64, 448)).astype(np.uint8)
    e8m0 = rng.integers(0, 256, (2, 64, 14)).astype(np.uint8)
    rope = rng.integers(0, 1 << 16, (2, 64, 64)).astype(np.uint16)
    buf, d = L.pack_kv_pool_fp4(codes, e8m0, rope, device="cpu")
    page = buf.numpy().reshape(2, 23552)
    nib = page[:, :14336].reshape(2, 64, 224)
    assert np.array_equal(nib & 15, codes[..., 0::2]) and np.array_equal(nib >> 4, codes[..., 1::2])
    assert np.array_equal(page[:, 14336:22528].copy().view(np.uint16).reshape(2, 64, 64), rope)
    assert np.array_equal(page[:, 22528:].reshape(2, 64, 16)[..., :14], e8m0)
    assert d.kind == L.POOL_KV_FP4 and d.num_pages == 2
