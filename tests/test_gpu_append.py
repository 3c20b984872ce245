"""Rows appended to the cache on the GPU against the oracle.

Without the norm the 448 nope values are quantised in fp32 from BF16 inputs on both sides: codes
and scales are compared bit for bit with the cache writer's oracle.  With it, y is fp32:
the mean of 512 squares, the root and the products are off by at most 2^-18 of y (as derived for
the rotated heads), so a scale is, and a code is one that lies nearest to y / scale give or take
2^-17 of it.  A rope value is two products and a sum in fp32, rounded once: 2^-8 of it and 2^-18
of the pair's magnitude.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv_fp4 import bf16_dev, bits_of, dev, random_pool, special_rows, unpack
from test_gpu_writer import rows_mix, unpack_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def table_of(L, rows):
    cs = torch.empty(rows, 32, 2, device="cuda")
    L.dsv4sa_rope_table(cs, base=160000.0, factor=16.0, original_len=65536)
    host = cs.double().cpu().numpy()
    return cs, host[..., 0] + 1j * host[..., 1]


def fp8_pool(rng, P):
    return {"nope_codes": rng.integers(0, 127, (P, 64, 448)).astype(np.uint8),
            "nope_scale": rng.uniform(0.1, 1, (P, 64, 7)).astype(np.float32),
            "rope_bits": bits_of(rng.standard_normal((P, 64, 64)))}


def device_pool(L, kind, pool):
    if kind == L.POOL_KV:
        return L.pack_kv_pool(pool["nope_codes"], pool["nope_scale"], pool["rope_bits"])
    return L.pack_kv_pool_fp4(pool["nope_codes"], pool["nope_e8m0"], pool["rope_bits"])


def host_pool(L, kind, buf, P):
    return unpack_kv(L, buf, P) if kind == L.POOL_KV else unpack(L, buf, P)[0]


def rope_ok(got_bits, y, mag):
    got = oracle.bf16_decode(got_bits)
    with np.errstate(invalid="ignore"):
        fine = np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * mag
    return fine | (np.isnan(got) & ~np.isfinite(y)) | (got == y)


def pair_mag(x):
    m = np.abs(x).reshape(32, 2).sum(1)
    return np.repeat(m, 2)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("n", [1, 5, 37, 700])
def test_unnormed_rows_are_the_writers(L, n, kind, rotate):
    rng = np.random.default_rng(50 + n + kind)
    P, B = 30, 3
    pool = fp8_pool(rng, P) if kind == L.POOL_KV else random_pool(rng, P)
    pt = rng.permutation(P)[:B * 9].reshape(B, 9).astype(np.int32)
    pairs = rng.permutation(B * 576)[:n]
    seq, ent = (pairs // 576).astype(np.int32), (pairs % 576).astype(np.int32)
    bits = bits_of(rows_mix(rng, n, 512)) if kind == L.POOL_KV else special_rows(rng, n)
    pos = rng.integers(0, 2000, n).astype(np.int32)
    cs, z = table_of(L, 2000)
    buf, desc = device_pool(L, kind, pool)
    L.dsv4sa_cache_append(desc, dev(pt), dev(seq), dev(pos) if rotate else None, bf16_dev(bits), cs if rotate else None,
                          row_entry=dev(ent))
    assert L.dsv4sa_check_errors() == (0, 0)
    got = host_pool(L, kind, buf, P)
    ref = {k: v.copy() for k, v in pool.items()}
    write = oracle.kv_write if kind == L.POOL_KV else oracle.kv_write_fp4
    for r in range(n):
        write(ref, pt[seq[r]], [ent[r]], bits[r:r + 1])
    for k in ref:
        if k == "rope_bits" and rotate:
            continue
        a, b = np.ascontiguousarray(got[k]).view(np.uint8), np.ascontiguousarray(ref[k]).view(np.uint8)
        assert (a == b).all(), (k, np.argwhere(a != b)[:4])
    if rotate:
        slots = {(int(pt[seq[r], ent[r] // 64]), int(ent[r] % 64)): r for r in range(n)}
        for pg in range(P):
            for sl in range(64):
                r = slots.get((pg, sl))
                if r is None:
                    assert (got["rope_bits"][pg, sl] == pool["rope_bits"][pg, sl]).all()
                    continue
                x = oracle.bf16_decode(bits[r])
                with np.errstate(invalid="ignore"):
                    y = oracle.append_row(bits[r], z[pos[r]])[448:]
                assert rope_ok(got["rope_bits"][pg, sl], y, pair_mag(x[448:])).all(), (r, pg, sl)




def nearest_ok(got, z, grid):
    """got is nearest to z on the grid, give or take 2^-17 of z (and of a denormal step)."""
    i = np.searchsorted(grid, got)
    assert (grid[i] == got).all()
    lo = np.where(i > 0, (grid[np.maximum(i - 1, 0)] + got) / 2, -np.inf)
    hi = np.where(i + 1 < grid.size, (grid[np.minimum(i + 1, grid.size - 1)] + got) / 2, np.inf)
    slack = 2.0 ** -17 * np.abs(z) + 1e-30
    return (z >= lo - slack) & (z <= hi + slack)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("kind", [0, 3])
@pytest.mark.parametrize("n,ring", [(1, 128), (40, 0), (65, 128)])
def test_normed_rows(L, n, ring, kind, weights):
    rng = np.random.default_rng(60 + n)
    P, B = 24, 5
    per = 2 if ring else 4
    pool = fp8_pool(rng, P) if kind == L.POOL_KV else random_pool(rng, P)
    pt = rng.permutation(P)[:B * per].reshape(B, per).astype(np.int32)
    seq = (np.arange(n) % B).astype(np.int32)
    pos = (rng.integers(0, 100 if not ring else 1900, B)[seq] + np.arange(n) // B).astype(np.int32)
    x = rng.standard_normal((n, 512)) * np.exp2(rng.integers(-20, 20, (n, 1))) * np.exp2(2 * rng.standard_normal(512))
    x[0, :64] = 0
    bits = bits_of(x)
    w = rng.uniform(0.25, 2, 512).astype(np.float32) if weights else None
    cs, z = table_of(L, 2000)
    buf, desc = device_pool(L, kind, pool)
    L.dsv4sa_cache_append(desc, dev(pt), dev(seq), dev(pos), bf16_dev(bits), cs, ring=ring, eps=1e-6,
                          norm_w=dev(w) if weights else None)
    assert L.dsv4sa_check_errors() == (0, 0)
    got = host_pool(L, kind, buf, P)
    written = np.zeros((P, 64), bool)
    e4m3 = np.unique(oracle.e4m3_decode(np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)))
    e2m1 = np.unique(oracle.e2m1_decode(np.arange(16, dtype=np.uint8)))
    for r in range(n):
        e = pos[r] % ring if ring else pos[r]
        pg, sl = pt[seq[r], e // 64], e % 64
        written[pg, sl] = True
        flat = oracle.append_row(bits[r], None, w, 1e-6)
        y = oracle.append_row(bits[r], z[pos[r]], w, 1e-6)
        assert rope_ok(got["rope_bits"][pg, sl], y[448:], pair_mag(flat[448:])).all()
        if kind == L.POOL_KV:
            blk = y[:448].reshape(7, 64)
            scale = np.maximum(np.abs(blk).max(1), 1e-4) / 448
            s = got["nope_scale"][pg, sl].astype(np.float64)
            assert (np.abs(s - scale) <= 2.0 ** -17 * scale).all()
            assert nearest_ok(oracle.e4m3_decode(got["nope_codes"][pg, sl]).reshape(7, 64), blk / scale[:, None], e4m3).all()
        else:
            blk = y[:448].reshape(14, 32)
            top = np.maximum(np.abs(blk).max(1), 6 * 2.0 ** -126) / 6
            b = got["nope_e8m0"][pg, sl].astype(np.int64) - 127
            # the smallest power of two at or above top, give or take 2^-17 of it
            assert (2.0 ** b >= top * (1 - 2.0 ** -17)).all() and (2.0 ** (b - 1) < top * (1 + 2.0 ** -17)).all()
            v = oracle.e2m1_decode(got["nope_codes"][pg, sl]).reshape(14, 32)
            assert nearest_ok(v, blk / 2.0 ** b[:, None], e2m1).all()
    for k in pool:
        a, c = np.ascontiguousarray(got[k][~written]).view(np.uint8), np.ascontiguousarray(pool[k][~written]).view(np.uint8)
        assert (a == c).all(), k


def test_strided_and_selected_rows(L):
    """Rows inside a wider projection, accepted ones picked by a list; row 3 twice, padding skipped."""
    rng = np.random.default_rng(70)
    P = 6
    wide = bf16_dev(bits_of(rng.standard_normal((9, 600))))
    rows = wide[:, 24:536]
    pt = np.array([[4, 1], [0, 3]], np.int32)
    seq = np.array([0, 1, -1, 1, 0], np.int32)
    ent = np.array([3, 70, -5, 0, 127], np.int32)
    src = np.array([8, 3, 999, 3, 0], np.int32)
    cs, _ = table_of(L, 300)
    pos = np.array([5, 299, -7, 0, 17], np.int32)
    pool = fp8_pool(rng, P)
    buf, desc = device_pool(L, L.POOL_KV, pool)
    L.dsv4sa_cache_append(desc, dev(pt), dev(seq), dev(pos), rows, cs, row_entry=dev(ent), src_row=dev(src))
    assert L.dsv4sa_check_errors() == (0, 0)
    want, wdesc = device_pool(L, L.POOL_KV, pool)
    live = [0, 1, 3, 4]
    L.dsv4sa_cache_append(wdesc, dev(pt), dev(seq[live]), dev(pos[live]), rows[torch.from_numpy(src[live]).long().cuda()].contiguous(), cs,
                          row_entry=dev(ent[live]))
    assert torch.equal(buf, want)


@pytest.mark.parametrize("kind", [0, 3])
def test_rows_out_of_range_are_flagged_and_skipped(L, kind):
    rng = np.random.default_rng(71)
    P = 4
    pool = fp8_pool(rng, P) if kind == L.POOL_KV else random_pool(rng, P)
    pt = np.array([[0, 9], [2, -1]], np.int32)
    cs, _ = table_of(L, 50)
    rows = bf16_dev(bits_of(rng.standard_normal((2, 512))))
    #        page id 9, entry past the table, negative entry, sequence -2, page id -1, position past the table, source row
    seq = [0, 0, 1, -2, 1, 1, 0]
    ent = [64, 128, -1, 0, 64, 3, 5]
    pos = [1, 1, 1, 1, 1, 50, 1]
    src = [0, 0, 1, 0, 1, 0, 2]
    for i in range(7):
        buf, desc = device_pool(L, kind, pool)
        before = buf.clone()
        L.dsv4sa_cache_append(desc, dev(pt), dev(np.array(seq[i:i + 1], np.int32)), dev(np.array(pos[i:i + 1], np.int32)), rows, cs,
                              row_entry=dev(np.array(ent[i:i + 1], np.int32)), src_row=dev(np.array(src[i:i + 1], np.int32)))
        assert L.dsv4sa_check_errors() == (5, 1), i
        assert torch.equal(buf, before), i


def test_graph_stream_and_empty(L):
    rng = np.random.default_rng(72)
    P, n = 8, 100
    pool = fp8_pool(rng, P)
    pt = np.arange(8, dtype=np.int32).reshape(4, 2)
    seq, pos = (np.arange(n) % 4).astype(np.int32), (np.arange(n) // 4 + 120).astype(np.int32)
    rows = bf16_dev(bits_of(rng.standard_normal((n, 512))))
    cs, _ = table_of(L, 200)
    args = (dev(pt), dev(seq), dev(pos), rows, cs)
    ref, rdesc = device_pool(L, L.POOL_KV, pool)
    L.dsv4sa_cache_append(rdesc, *args, ring=128, eps=1e-6)
    buf, desc = device_pool(L, L.POOL_KV, pool)
    start = buf.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.dsv4sa_cache_append(desc, *args, ring=128, eps=1e-6)
    for _ in range(2):
        buf.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, ref)
    buf.copy_(start)
    s.wait_stream(torch.cuda.current_stream())
    L.dsv4sa_cache_append(desc, *args, ring=128, eps=1e-6, stream=s)
    s.synchronize()
    assert torch.equal(buf, ref)
    L.dsv4sa_cache_append(desc, args[0], args[1][:0], args[2][:0], rows[:0], cs, ring=128)
    assert L.dsv4sa_check_errors() == (0, 0)
