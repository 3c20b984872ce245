"""The FP4 cache in the framework's own serving paths (run_path, StepGraph, NativeStep),
beside rows that are no numbers, and the pages' calls captured into graphs and run on
several streams at once."""
import numpy as np
import pytest
import torch

import oracle
from compressed_sparse_attention_c4_gb300 import workloads as W
from test_gpu_kv_fp4 import SCALE, Case, attention_reference, dev, unpack
from test_gpu_pages import Cache, i32, sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def test_requantised_pool(L):
    """Every page of an FP8 pool, read as BF16 (value rounded once) and quantised to FP4."""
    w = W.make("tiny")
    d8, d4 = L.upload(w), L.upload(w, kv_fp4=True)
    assert d4.comp.kind == d4.win.kind == L.POOL_KV_FP4 and d4.attn_ws is None
    P = int(d8.comp.num_pages)
    entries = np.arange(P * 64)
    rows = oracle.kv_rows(w.comp_pool, np.arange(P), entries)
    bits = torch.from_numpy(rows).float().to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    ref = {"nope_codes": np.zeros((P, 64, 448), np.uint8), "nope_e8m0": np.zeros((P, 64, 14), np.uint8),
           "rope_bits": np.zeros((P, 64, 64), np.uint16)}
    oracle.kv_write_fp4(ref, np.arange(P), entries, bits)
    got, _ = unpack(L, d4.comp_buf, P)
    for k in ref:
        assert np.array_equal(got[k], ref[k]), k


@pytest.mark.parametrize("name", ["tiny", "decode"])
def test_serving_steps_over_fp4_pools(L, name):
    """run_path over FP4 pools against the oracle; the graph of it and the step built by
    the library give its bits, launch after launch, and follow new inputs."""
    w = W.make(name)
    d = L.upload(w, kv_fp4=True)
    L.run_path(d, fused_window=True)
    torch.cuda.synchronize()
    assert L.dsv4sa_check_errors() == (0, 0)
    out, lse = d.out.float().cpu().numpy(), d.lse.cpu().numpy()
    comp, _ = unpack(L, d.comp_buf, int(d.comp.num_pages))
    win, _ = unpack(L, d.win_buf, int(d.win.num_pages))
    idx = d.idx_c.cpu().numpy()
    scale = float(w.softmax_scale)
    assert abs(scale - SCALE) < 1e-12                            # the reference's bounds take this scale
    for t in sorted({0, w.T // 2, w.T - 1}):
        s = int(w.q_seq[t])
        kv = oracle.gather_rows_fp4(idx[t], comp, w.comp_pt[s], oracle.window_indices(int(w.pos[t]), w.kw, w.win_ring), win, w.win_pt[s])
        o, l, tol, ltol = attention_reference(np.ascontiguousarray(w.q[t]).view(np.uint16), np.asarray(w.sink, np.float32), kv)
        assert (np.abs(out[t] - o) <= tol).all() and (np.abs(lse[t] - l) <= ltol).all()
    for make in (L.StepGraph, L.NativeStep):
        step = make(d)
        go = step.replay if make is L.StepGraph else step.launch
        for _ in range(2):
            step.host_out["out"].fill_(7.0)
            go()
            step.stream.synchronize()
            assert np.array_equal(step.host_out["out"].float().numpy(), out)
            assert np.array_equal(step.host_out["lse"].numpy(), lse)
        q = step.host_in["q"].clone()
        step.host_in["q"].view(torch.int16).fill_(0x3F80)        # every query element 1.0: a different softmax
        go()
        step.stream.synchronize()
        other = step.host_out["out"].float().numpy()
        assert np.isfinite(other).all() and np.abs(other - out).max() > 0.05 * np.abs(out).max()
        step.host_in["q"].copy_(q)
        go()
        step.stream.synchronize()
        assert np.array_equal(step.host_out["out"].float().numpy(), out)
        if make is L.NativeStep:
            step.close()
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("H,T", [(16, 1), (64, 3), (64, 170), (40, 20)])
def test_rows_that_no_list_names_may_hold_anything(L, H, T):
    """NaN and infinities in every slot that is not attended to change no bit; in a slot
    that one query attends to they stay in that query."""
    c = Case(L, T, H, 200, 64, seed=77, ring=64, entries=900)
    fn = L.dsv4sa_sparse_attn_decode
    out, lse = c.run(L, fn)
    named = {"comp": np.zeros((c.comp["nope_codes"].shape[0], 64), bool), "win": np.zeros((c.win["nope_codes"].shape[0], 64), bool)}
    for t in range(T):
        s = c.seq[t]
        for key, e, pt in (("comp", c.idx[t], c.comp_pt[s]), ("win", c.window(t), c.win_pt[s])):
            e = np.asarray(e)[np.asarray(e) >= 0]
            named[key][pt[e // 64], e % 64] = True
    for key, pool in (("comp", c.comp), ("win", c.win)):
        free = ~named[key]
        pool["nope_e8m0"][free] = 255
        pool["rope_bits"][free] = 0x7FC0
        pool["rope_bits"][free, ::2] = 0xFF80
    for key, buf in (("comp", c.comp_buf), ("win", c.win_buf)):
        p = getattr(c, key)
        buf.copy_(L.pack_kv_pool_fp4(p["nope_codes"], p["nope_e8m0"], p["rope_bits"])[0])
    again, lse2 = c.run(L, fn)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    free = np.argwhere(~named["comp"])
    if T > 1 and len(free):
        t = T // 2                                               # an entry of its sequence that nobody names
        s = int(c.seq[t])
        mine = [(j * 64 + sl) for j, pg in enumerate(c.comp_pt[s]) for sl in np.flatnonzero(~named["comp"][pg])]
        if mine:
            c.d["idx"][t, 0] = mine[0]
            bad, _ = c.run(L, fn)
            assert torch.isnan(bad[t]).all()
            keep = [i for i in range(T) if i != t]
            assert torch.equal(bad[keep], out[keep])
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("T,H,kc", [(1, 16, 2048), (8, 16, 500), (32, 16, 500), (64, 16, 1000), (3, 40, 2048), (4, 64, 2048),
                                    (16, 64, 500), (32, 64, 500), (64, 64, 500), (32, 64, 2048), (64, 64, 2048), (130, 64, 2048),
                                    (5, 128, 130), (200, 20, 300)])
def test_every_split_of_heads_and_rows(L, T, H, kc):
    """Batches and lists over which the work is dealt out differently: items of 16, 32 and
    64 heads, alone or over clusters of 2, 4 and 8 (and several items a CTA)."""
    c = Case(L, T, H, kc, 128, seed=T + H + kc, ring=128, entries=3000, empty=(T // 3,))
    out, lse = c.run(L, L.dsv4sa_sparse_attn_decode)
    assert L.dsv4sa_check_errors() == (0, 0)
    c.check(out, lse, rows=sorted({0, 1 % T, T // 3, T // 2, T - 1}))
    pre, lse_p = c.run(L, L.dsv4sa_sparse_attn_prefill)         # never over clusters
    c.check(pre, lse_p, rows=sorted({0, T // 3, T - 1}))
    # everywhere: the two differ by no more than their bounds, 2^-6 of the largest value being far above both
    assert (out.double() - pre.double()).abs().max() <= 2.0 ** -6 * float(out.abs().max())
    assert (lse.double() - lse_p.double()).abs().max() <= 2.0 ** -12 * float(lse.abs().max().clamp(min=1.0))


def test_long_window_without_a_list_and_long_sequences(L):
    """Entries far up a sequence: page-table columns past 2^15, entries past 2^21."""
    rng = np.random.default_rng(4)
    T, H, kc, stride = 2, 16, 300, 40000
    c = Case(L, T, H, kc, 0, seed=11)
    P = c.comp["nope_codes"].shape[0]
    table = torch.randint(0, P, (2, stride), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    idx = rng.integers(stride * 64 - 500000, stride * 64, (T, kc)).astype(np.int32)
    c.comp_pt, c.idx = table.numpy(), idx
    c.d["comp_pt"], c.d["idx"] = table.cuda(), dev(idx)
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        c.check(*c.run(L, fn))
    assert L.dsv4sa_check_errors() == (0, 0)


# ---------------------------------------------------------------- pages in graphs and streams

def beam_cache(L, seed, pages=64):
    return Cache(L, (L.POOL_KV_FP4, L.POOL_IDXK_FP4), pages, 9, 6, seed=seed,
                 fill=sequences([200, 64, 1], 9, 6, pages))


def test_release_fork_compact_in_a_graph(L):
    """One graph of a beam step, replayed: rows released, forks of rows that the replay
    before made, the cache compacted in place."""
    c = beam_cache(L, 5)
    table, use, pools = c.table.copy(), c.use.copy(), c.pools()
    drop, src, dst = i32([3, 4, 5]), i32([0, 0, 2]), i32([3, 4, 5])
    length, new = i32([200, 190, 1]), torch.empty(3, dtype=torch.int32, device="cuda")
    new_id, n_used = torch.empty(c.P, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")

    def body():
        L.dsv4sa_cache_release(c.cache, drop)
        L.dsv4sa_cache_fork(c.cache, src, dst, length, new)
        L.dsv4sa_cache_compact(c.cache, c.cache, new_id, n_used)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        body()
    c.same(table, use, pools)                                    # capturing ran nothing
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        oracle.cache_release(table, use, [3, 4, 5])
        want = oracle.cache_fork(table, use, pools, [0, 0, 2], [3, 4, 5], [200, 190, 1])
        assert new.cpu().numpy().tolist() == want.tolist()
        ids = oracle.cache_compact_ids(use, True)
        assert np.array_equal(new_id.cpu().numpy(), ids) and int(n_used) == int((use > 0).sum())
        moved = np.flatnonzero((ids >= 0) & (ids != np.arange(c.P)))
        for p in pools:
            p[ids[moved]] = p[moved]
        table[:] = np.where(table >= 0, ids[np.maximum(table, 0)], -1)
        use[:] = oracle.use_counts(table, c.P)
        c.same(table, use, pools)
        length.copy_(i32([130, 192, 1]))                         # the next replay reads the new lengths
        g.replay()
        torch.cuda.synchronize()
        oracle.cache_release(table, use, [3, 4, 5])
        oracle.cache_fork(table, use, pools, [0, 0, 2], [3, 4, 5], [130, 192, 1])
        ids = oracle.cache_compact_ids(use, True)
        moved = np.flatnonzero((ids >= 0) & (ids != np.arange(c.P)))
        for p in pools:
            p[ids[moved]] = p[moved]
        table[:] = np.where(table >= 0, ids[np.maximum(table, 0)], -1)
        use[:] = oracle.use_counts(table, c.P)
        c.same(table, use, pools)
        length.copy_(i32([200, 190, 1]))
    assert L.dsv4sa_check_errors() == (0, 0)


def test_two_caches_on_two_streams(L):
    """Different caches at once: neither call has state that the other shares."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [beam_cache(L, 20 + i, pages=4000) for i in range(2)]
    want = []
    for c in caches:
        table, use, pools = c.table.copy(), c.use.copy(), c.pools()
        new = oracle.cache_fork(table, use, pools, [0, 1, 2, 0], [3, 4, 5, 6], [200, 64, 1, 65])
        oracle.cache_release(table, use, [0, 5])
        want.append((table, use, pools, new))
    args = [(i32([0, 1, 2, 0]), i32([3, 4, 5, 6]), i32([200, 64, 1, 65]), torch.empty(4, dtype=torch.int32, device="cuda"), i32([0, 5]))
            for _ in caches]
    torch.cuda.synchronize()
    for c, a, s in zip(caches, args, streams):
        with torch.cuda.stream(s):
            L.dsv4sa_cache_fork(c.cache, *a[:4])
            L.dsv4sa_cache_release(c.cache, a[4])
    torch.cuda.synchronize()
    for c, a, (table, use, pools, new) in zip(caches, args, want):
        c.same(table, use, pools)
        assert a[3].cpu().numpy().tolist() == new.tolist()
    assert L.dsv4sa_check_errors() == (0, 0)


def test_fork_copies_a_hole_as_a_hole(L):
    """An entry of the parent that is no page, before its last: -1 in the child, flagged."""
    c = beam_cache(L, 8)
    c.table[0, 1] = -1
    c.use = oracle.use_counts(c.table, c.P)
    c.upload()
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    L.dsv4sa_cache_fork(c.cache, i32([0]), i32([3]), i32([192]), new)
    assert L.dsv4sa_check_errors() == (5, 1)
    table = c.d_table.cpu().numpy()
    assert table[3].tolist() == [c.table[0, 0], -1, c.table[0, 2], -1, -1, -1] and int(new) == -1
    assert np.array_equal(c.d_use.cpu().numpy(), oracle.use_counts(table, c.P))
