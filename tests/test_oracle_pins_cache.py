"""The oracle's FP4 KV cache, pages and norm, pinned against values that do not come
from it: hand codes, torch's decoders and casts, brute-force loops, invariants."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from oracle import dsv4sa_oracle as oracle                      # noqa: E402

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]                 # the format's magnitudes
E2M1 = np.array(E2M1 + [-v for v in E2M1])


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def bf16_values(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).double().numpy()


def empty_pool(pages):
    return {"nope_codes": np.full((pages, 64, 448), 9, np.uint8), "nope_e8m0": np.full((pages, 64, 14), 3, np.uint8),
            "rope_bits": np.full((pages, 64, 64), 7, np.uint16)}


def test_kv_write_fp4_hand_block():
    """A block of the format's own values times 2^3: the scale is 2^3 and every code is hit."""
    pool, row = empty_pool(2), np.zeros(512, np.float32)
    row[:32] = np.tile(E2M1, 2) * 8.0
    row[448:] = np.arange(64)
    oracle.kv_write_fp4(pool, np.array([1]), np.array([5]), bf16_bits(row)[None])
    # -0 keeps its sign bit or not: the value is what counts
    assert np.array_equal(E2M1[pool["nope_codes"][1, 5, :32]], np.tile(E2M1, 2))
    assert pool["nope_e8m0"][1, 5, 0] == 130
    assert np.array_equal(bf16_values(pool["rope_bits"][1, 5]), np.arange(64.0))
    got = oracle.kv_rows_fp4(pool, np.array([1]), np.array([5]))[0]
    assert np.array_equal(got, row.astype(np.float64))
    keep = np.ones((2, 64), bool)
    keep[1, 5] = False
    for k, v in empty_pool(2).items():
        assert np.array_equal(pool[k][keep], v[keep])            # nothing else is written


def test_kv_write_fp4_blocks_with_no_number():
    for bad in (np.inf, -np.inf, np.nan):
        pool, row = empty_pool(1), np.ones(512, np.float32)
        row[40] = bad
        row[500] = bad
        oracle.kv_write_fp4(pool, np.array([0]), np.array([0]), bf16_bits(row)[None])
        got = oracle.kv_rows_fp4(pool, np.array([0]), np.array([0]))[0]
        assert np.isnan(got[32:64]).all() and np.isfinite(np.delete(got[:448], np.arange(32, 64))).all()
        assert got[500] == bad or (np.isnan(bad) and np.isnan(got[500]))     # rope as stored


def test_kv_rows_fp4_brute_force():
    rng = np.random.default_rng(5)
    pool = {"nope_codes": rng.integers(0, 16, (3, 64, 448)).astype(np.uint8),
            "nope_e8m0": rng.integers(0, 255, (3, 64, 14)).astype(np.uint8),
            "rope_bits": bf16_bits(rng.standard_normal((3, 64, 64)))}
    pt, entries = np.array([2, 0, 1]), np.array([0, 63, 64, 130, 191])
    got = oracle.kv_rows_fp4(pool, pt, entries)
    for r, e in enumerate(entries):
        pg, sl = pt[e // 64], e % 64
        want = [E2M1[pool["nope_codes"][pg, sl, d]] * 2.0 ** (int(pool["nope_e8m0"][pg, sl, d // 32]) - 127) for d in range(448)]
        assert np.array_equal(got[r, :448], want)
        assert np.array_equal(got[r, 448:], bf16_values(pool["rope_bits"][pg, sl]))


def test_kv_write_fp4_error_bound():
    """Round to nearest in blocks of 32: off by at most half the grid's step."""
    rng = np.random.default_rng(6)
    rows = bf16_bits(rng.standard_normal((64, 512)) * np.exp2(rng.integers(-30, 30, (64, 1))))
    pool = empty_pool(1)
    oracle.kv_write_fp4(pool, np.array([0]), np.arange(64), rows)
    got, x = oracle.kv_rows_fp4(pool, np.array([0]), np.arange(64)), bf16_values(rows)
    scale = np.repeat(np.exp2(pool["nope_e8m0"][0].astype(np.float64) - 127), 32, axis=1)
    y = np.abs(x[:, :448]) / scale
    assert y.max() <= 6.0
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
    assert np.all(np.abs(got[:, :448] - x[:, :448]) <= half * scale)
    assert np.array_equal(got[:, 448:], x[:, 448:])


def test_gather_rows_fp4_is_kv_rows_of_the_valid_entries():
    rng = np.random.default_rng(7)
    pools = [{"nope_codes": rng.integers(0, 16, (2, 64, 448)).astype(np.uint8),
              "nope_e8m0": rng.integers(110, 140, (2, 64, 14)).astype(np.uint8),
              "rope_bits": bf16_bits(rng.standard_normal((2, 64, 64)))} for _ in range(2)]
    c, w = np.array([3, -1, 100, 3]), np.array([-1, 64])
    got = oracle.gather_rows_fp4(c, pools[0], np.array([1, 0]), w, pools[1], np.array([0, 1]))
    assert got.shape == (4, 512)
    assert np.array_equal(got[:3], oracle.kv_rows_fp4(pools[0], np.array([1, 0]), np.array([3, 100, 3])))
    assert np.array_equal(got[3:], oracle.kv_rows_fp4(pools[1], np.array([0, 1]), np.array([64])))
    assert oracle.gather_rows_fp4(None, None, None, np.array([-1, -1]), pools[1], np.array([0, 1])).shape == (0, 512)


@pytest.mark.parametrize("group", [64, 128])
def test_rms_norm_quant(group):
    rng = np.random.default_rng(8)
    x, r = bf16_bits(rng.standard_normal((5, 256))), bf16_bits(rng.standard_normal((5, 256)))
    w = rng.uniform(0.5, 1.5, 256).astype(np.float32)
    got = oracle.rms_norm_quant(x, r, w, 1e-6, group)
    s = torch.from_numpy(bf16_values(x) + bf16_values(r))
    y = torch.nn.functional.rms_norm(s, (256,), torch.from_numpy(w).double(), 1e-6)
    np.testing.assert_allclose(got["s"], s.numpy(), rtol=0, atol=0)
    np.testing.assert_allclose(got["y"], y.numpy(), rtol=1e-14)
    amax = np.abs(y.numpy()).reshape(5, -1, group).max(-1)
    np.testing.assert_allclose(got["scale"], amax / 448.0, rtol=1e-14)
    assert abs(np.abs(got["z"]).max() - 448.0) < 1e-9
    np.testing.assert_allclose(got["z"] * np.repeat(got["scale"], group, axis=1), y.numpy(), rtol=1e-14)
    alone = oracle.rms_norm_quant(x, None, w, 1e-6, group)
    assert np.array_equal(alone["s"], bf16_values(x))


def test_rms_norm_quant_of_zeros_has_the_floor_scale():
    got = oracle.rms_norm_quant(np.zeros((1, 128), np.uint16), None, np.ones(128, np.float32), 1e-6, 128)
    assert got["scale"][0, 0] == 1e-4 / 448.0 and not got["z"].any()


def agree(table, use):
    assert np.array_equal(oracle.use_counts(table, len(use)), use)


def test_fork_and_release_hand_case():
    # row 0 holds 150 slots in pages 3, 0, 4; pages 1, 2, 5 are free
    table = np.array([[3, 0, 4], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    use = np.array([1, 0, 0, 1, 1, 0], np.int32)
    data = np.arange(6 * 64).reshape(6, 64).copy()
    before = data.copy()
    new = oracle.cache_fork(table, use, [data], [0, 0, 0], [1, 2, 3], [150, 128, 65])
    assert new.tolist() == [1, -1, 2]
    assert table[1].tolist() == [3, 0, 1] and table[2].tolist() == [3, 0, -1] and table[3].tolist() == [3, 2, -1]
    assert use.tolist() == [3, 1, 1, 4, 1, 0]
    agree(table, use)
    assert np.array_equal(data[1, :22], before[4, :22]) and np.array_equal(data[1, 22:], before[1, 22:])
    assert np.array_equal(data[2, :1], before[0, :1]) and np.array_equal(data[2, 1:], before[2, 1:])
    assert np.array_equal(data[[0, 3, 4, 5]], before[[0, 3, 4, 5]])
    assert oracle.cache_fork(table, use, [data], [0, 0], [4, 5], [10, 10]).tolist() == [5, -2]   # one page left
    assert table[5].tolist() == [-1, -1, -1]
    agree(table, use)
    oracle.cache_release(table, use, [0, -1, 0, 2])
    assert use.tolist() == [1, 1, 1, 2, 0, 1] and (table[[0, 2]] == -1).all()
    agree(table, use)


def test_compact_ids():
    use = np.array([0, 2, 0, 1, 0, 1, 3], np.int32)
    assert oracle.cache_compact_ids(use, False).tolist() == [-1, 0, -1, 1, -1, 2, 3]
    assert oracle.cache_compact_ids(use, True).tolist() == [-1, 1, -1, 3, -1, 0, 2]
    rng = np.random.default_rng(9)
    for n in (1, 2, 63, 200):
        u = (rng.random(n) < 0.5).astype(np.int32)
        for in_place in (False, True):
            ids = oracle.cache_compact_ids(u, in_place)
            assert sorted(ids[u > 0]) == list(range(int(u.sum()))) and (ids[u == 0] == -1).all()
            if in_place:
                moved = (ids >= 0) & (ids != np.arange(n))
                assert all(u[i] == 0 for i in ids[moved])        # into free pages only
