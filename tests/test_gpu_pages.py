"""Pages of a cache on the GPU (dsv4sa_pages_copy, dsv4sa_cache_fork, _release, _compact):
tables, counts, ids and every byte of every pool equal the oracle's."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


class Cache:
    """Pools of the given kinds with random bytes, random rows, counts that agree."""

    def __init__(self, L, kinds, pages, rows, stride, seed=0, fill=None):
        rng = np.random.default_rng(seed)
        self.L, self.kinds, self.P = L, kinds, pages
        self.bufs = [L._alloc_pool(k, pages, "cuda") for k in kinds]
        self.descs = [L.dsv4sa_pool_desc_init(k, b, pages) for k, b in zip(kinds, self.bufs)]
        for b in self.bufs:
            b.copy_(torch.from_numpy(rng.integers(0, 256, b.numel()).astype(np.uint8)))
        self.table = np.full((rows, stride), -1, np.int32)
        if fill is not None:
            self.table[:] = fill(rng)
        self.use = oracle.use_counts(self.table, pages)
        self.upload()

    def upload(self):
        self.d_table, self.d_use = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.use).cuda()
        self.cache = self.L.page_cache(self.descs, self.d_table, self.d_use)

    def pools(self):
        """Logical arrays: one [P, 64, bytes per slot] array per block of each pool."""
        out = []
        for d, b in zip(self.descs, self.bufs):
            host = b.cpu().numpy().reshape(self.P, d.page_stride)
            for off, row in ((d.nope_off, d.nope_row), (d.rope_off, d.rope_row), (d.scale_off, d.scale_row)):
                if row:
                    out.append(host[:, off:off + 64 * row].reshape(self.P, 64, row).copy())
        return out

    def same(self, table, use, pools):
        np.testing.assert_array_equal(self.d_table.cpu().numpy(), table)
        np.testing.assert_array_equal(self.d_use.cpu().numpy(), use)
        for a, b in zip(self.pools(), pools):
            np.testing.assert_array_equal(a, b)


def i32(x):
    return torch.tensor(np.asarray(x, np.int32)).cuda()


KIND_SETS = [(0, 1), (3, 2), (3,), (0, 1, 2, 3)]


def sequences(lengths, rows, stride, pages):
    def fill(rng):
        t = np.full((rows, stride), -1, np.int32)
        perm = rng.permutation(pages)
        at = 0
        for r, n in enumerate(lengths):
            k = -(-n // 64)
            t[r, :k] = perm[at:at + k]
            at += k
        return t
    return fill


@pytest.mark.parametrize("kinds", KIND_SETS)
def test_copy(L, kinds):
    c = Cache(L, kinds, 40, 2, 4, seed=1)
    src = [3, 5, -1, 7, 9, 3]
    dst = [10, 11, 12, -1, 9, 39]                # skipped pairs, a page onto itself, one source twice
    want = c.pools()
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            for p in want:
                p[b] = p[a]
    L.dsv4sa_pages_copy(c.descs, i32(src), i32(dst))
    assert L.dsv4sa_check_errors() == (0, 0)
    c.same(c.table, c.use, want)
    L.dsv4sa_pages_copy(c.descs, i32([40, 2, -5]), i32([1, 41, 2]))
    assert L.dsv4sa_check_errors() == (5, 1)
    c.same(c.table, c.use, want)


@pytest.mark.parametrize("kinds", KIND_SETS)
@pytest.mark.parametrize("width", [1, 3, 40])
def test_fork_and_release(L, kinds, width):
    lengths = [0, 1, 63, 64, 65, 200, 256]
    rows = len(lengths) * (1 + width)
    pages = 17 + len(lengths) * width
    c = Cache(L, kinds, pages, rows, 6, seed=width, fill=sequences(lengths, rows, 6, pages))
    rng = np.random.default_rng(7)
    src = np.repeat(np.arange(len(lengths)), width)[rng.permutation(len(lengths) * width)].astype(np.int32)
    dst = np.arange(len(lengths), rows, dtype=np.int32)
    length = np.array([lengths[s] for s in src], np.int32)
    length[::5] = np.maximum(length[::5] - 30, 0)          # a prefix of the parent
    table, use, pools = c.table.copy(), c.use.copy(), c.pools()
    new = torch.full((len(src),), 77, dtype=torch.int32, device="cuda")
    L.dsv4sa_cache_fork(c.cache, i32(src), i32(dst), i32(length), new)
    assert L.dsv4sa_check_errors() == (0, 0)
    want = oracle.cache_fork(table, use, pools, src, dst, length)
    np.testing.assert_array_equal(new.cpu().numpy(), want)
    np.testing.assert_array_equal(use, oracle.use_counts(table, pages))
    c.same(table, use, pools)
    # parents and some forks go, one row named twice, one skipped, an empty row
    gone = list(range(len(lengths))) + list(dst[::2]) + [int(dst[0]), -1]
    L.dsv4sa_cache_release(c.cache, i32(gone))
    assert L.dsv4sa_check_errors() == (0, 0)
    oracle.cache_release(table, use, dict.fromkeys(gone))
    np.testing.assert_array_equal(use, oracle.use_counts(table, pages))
    c.same(table, use, pools)


def test_fork_takes_the_lowest_free_pages_far_into_the_pool(L):
    """Free pages beyond the first 8192 counts, more forks than threads of a CTA."""
    pages, n = 20000, 1500
    c = Cache(L, (2,), pages, n + 1, 2, seed=3)
    c.table[0, 0] = 11
    c.use[:] = 1
    free = np.random.default_rng(5).permutation(pages)[:n + 20]
    free = free[(free != 11)]
    c.use[free] = 0
    c.upload()
    new = torch.empty(n, dtype=torch.int32, device="cuda")
    pools = c.pools()
    L.dsv4sa_cache_fork(c.cache, i32(np.zeros(n)), i32(np.arange(1, n + 1)), i32(np.arange(n) % 63 + 1), new)
    assert L.dsv4sa_check_errors() == (0, 0)
    want = np.sort(free)[:n]
    np.testing.assert_array_equal(new.cpu().numpy(), want)
    for p in pools:
        for i, q in enumerate(want):
            p[q, :i % 63 + 1] = p[11, :i % 63 + 1]
    for a, b in zip(c.pools(), pools):
        np.testing.assert_array_equal(a, b)


def test_refused_forks(L):
    pages = 12
    c = Cache(L, (3, 2), pages, 8, 3, seed=4, fill=sequences([100, 64, 30], 8, 3, pages))
    c.table[6, 0] = 9                                       # a row in use
    c.use = oracle.use_counts(c.table, pages)
    c.upload()
    table, use, pools = c.table.copy(), c.use.copy(), c.pools()
    new = torch.empty(9, dtype=torch.int32, device="cuda")
    #        in use  row out  itself  len out  empty src  taken twice (second refused)  a dst as src
    src = [0, 0, 0, 1, 7, 0, 1, 3, -1]
    dst = [6, 8, 0, 4, 5, 3, 3, 7, 4]
    length = [100, 100, 100, 193, 5, 100, 64, 70, 10]
    L.dsv4sa_cache_fork(c.cache, i32(src), i32(dst), i32(length), new)
    assert L.dsv4sa_check_errors() == (5, 1)
    want = oracle.cache_fork(table, use, pools, [0], [3], [100])
    np.testing.assert_array_equal(new.cpu().numpy(), [-3, -3, -3, -3, -3, want[0], -3, -3, -3])
    c.same(table, use, pools)
    # no free page left: the first forks get theirs, the others' rows stay empty
    c.d_use[c.d_use == 0] = 1
    c.d_use[5 if use[5] == 0 else int(np.flatnonzero(use == 0)[0])] = 0
    use = c.d_use.cpu().numpy().copy()
    new = torch.empty(3, dtype=torch.int32, device="cuda")
    L.dsv4sa_cache_fork(c.cache, i32([2, 2, 1]), i32([4, 5, 7]), i32([30, 29, 64]), new)
    assert L.dsv4sa_check_errors() == (7, 4)
    want = oracle.cache_fork(table, use, pools, [2, 2, 1], [4, 5, 7], [30, 29, 64])
    assert want[1] == -2 and want[2] == -1
    np.testing.assert_array_equal(new.cpu().numpy(), want)
    c.same(table, use, pools)


def test_release_flags_what_it_cannot_count_down(L):
    c = Cache(L, (1,), 10, 4, 3, seed=6, fill=lambda rng: [[1, 2, -1], [2, 3, -1], [5, 6, -1], [-1, -1, -1]])
    c.d_table[1, 1] = 40                                    # a page id out of range
    c.d_use[5] = 0                                          # a page that is free already
    L.dsv4sa_cache_release(c.cache, i32([0, 1, 2, 4, -2]))
    assert L.dsv4sa_check_errors() == (5, 1)
    assert (c.d_table.cpu().numpy() == -1).all()
    np.testing.assert_array_equal(c.d_use.cpu().numpy(), [0, 0, 0, 1, 0, 0, 0, 0, 0, 0])


def fragmented(pages, rows, stride, used, seed):
    def fill(rng):
        t = np.full(rows * stride, -1, np.int32)
        ids = rng.permutation(pages)[:used]
        t[:used] = ids
        more = min(rows * stride - used, used // 3)
        t[used:used + more] = ids[:more]                    # shared pages
        return rng.permutation(t).reshape(rows, stride)
    return fill


@pytest.mark.parametrize("pages,used", [(1, 1), (1, 0), (9, 4), (100, 37), (100, 100), (8191, 4000), (20011, 16000), (20011, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(L, pages, used, in_place):
    kinds = (2,) if pages > 5000 else (3, 1)
    rows, stride = 7, used // 5 + 2
    c = Cache(L, kinds, pages, rows, stride, seed=pages + used, fill=fragmented(pages, rows, stride, used, 0))
    new_id = torch.full((pages,), 55, dtype=torch.int32, device="cuda")
    n_used = torch.full((1,), 55, dtype=torch.int32, device="cuda")
    before = c.pools()
    want = oracle.cache_compact_ids(c.use, in_place)
    moved = np.flatnonzero(want >= 0)
    table = np.where(c.table >= 0, want[np.maximum(c.table, 0)], -1)
    if in_place:
        L.dsv4sa_cache_compact(c.cache, c.cache, new_id, n_used)
        after, dst = c, [p.copy() for p in before]
        use = np.zeros(pages, np.int32)
    else:
        after = Cache(L, kinds, used + 2, rows, stride, seed=99)
        dst = after.pools()
        use = np.zeros(used + 2, np.int32)
        L.dsv4sa_cache_compact(c.cache, after.cache, new_id, n_used)
    assert L.dsv4sa_check_errors() == (0, 0)
    for a, b in zip(dst, before):
        a[want[moved]] = b[moved]
    use[want[moved]] = c.use[moved]
    assert int(n_used) == used
    np.testing.assert_array_equal(new_id.cpu().numpy(), want)
    after.same(table, use, dst)
    np.testing.assert_array_equal(use, oracle.use_counts(table, len(use)))
    if not in_place:
        c.same(c.table, c.use, before)                      # the source is left as it was


def test_compact_into_too_few_pages(L):
    c = Cache(L, (2,), 50, 3, 10, seed=2, fill=fragmented(50, 3, 10, 20, 0))
    d = Cache(L, (2,), 12, 3, 10, seed=3)
    new_id, n_used = torch.empty(50, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    before, dst = c.pools(), d.pools()
    L.dsv4sa_cache_compact(c.cache, d.cache, new_id, n_used)
    assert L.dsv4sa_check_errors() == (7, 4)
    want = oracle.cache_compact_ids(c.use, False)
    want[want >= 12] = -1
    np.testing.assert_array_equal(new_id.cpu().numpy(), want)
    moved = np.flatnonzero(want >= 0)
    for a, b in zip(dst, before):
        a[want[moved]] = b[moved]
    d.same(np.where(c.table >= 0, want[np.maximum(c.table, 0)], -1), c.use[moved], dst)


def test_a_decode_loop_with_beams_over_an_fp4_cache(L):
    """Together, as they would be used: rows written, forked, written apart, attended
    to, released, compacted and attended to again, every result against the oracle."""
    rng = np.random.default_rng(17)
    P, H, rows, stride = 24, 16, 6, 4
    c = Cache(L, (L.POOL_KV_FP4, L.POOL_IDXK_FP4), P, rows, stride, seed=1)
    kv = c.descs[0]
    # row 0: 100 entries on pages 20, 3; rows 1-3 fork it
    c.table[0, :2] = [20, 3]
    c.use = oracle.use_counts(c.table, P)
    c.upload()

    def write(table, row, entries, x):
        L.dsv4sa_cache_write(kv, table, i32(np.full(len(entries), row)), i32(entries), x)

    x0 = torch.randn(100, 512, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    write(c.d_table, 0, np.arange(100), x0)
    new = torch.empty(3, dtype=torch.int32, device="cuda")
    L.dsv4sa_cache_fork(c.cache, i32([0, 0, 0]), i32([1, 2, 3]), i32([100, 100, 64]), new)
    values = {r: [x0] for r in range(3)}
    values[3] = [x0[:64]]
    for r in range(3):                                     # each beam goes on with rows of its own
        xs = torch.randn(20, 512, generator=torch.Generator().manual_seed(10 + r)).to(torch.bfloat16).cuda()
        write(c.d_table, r, np.arange(100, 120), xs)
        values[r].append(xs)

    def attend(descs, table, live):
        T = len(live)
        q = torch.randn(T, H, 512, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
        idx = torch.full((T, 128), -1, dtype=torch.int32, device="cuda")
        for i, r in enumerate(live):
            n = sum(v.shape[0] for v in values[r])
            idx[i, :n] = torch.arange(n, dtype=torch.int32)
        out, sink = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, device="cuda")
        L.dsv4sa_sparse_attn_decode(q, sink, i32(live), descs[0], table, idx, None, None, None, out, 512 ** -0.5)
        assert L.dsv4sa_check_errors() == (0, 0)
        for i, r in enumerate(live):
            x = torch.cat(values[r]).cpu()
            pool = {"nope_codes": np.zeros((2, 64, 448), np.uint8), "nope_e8m0": np.zeros((2, 64, 14), np.uint8),
                    "rope_bits": np.zeros((2, 64, 64), np.uint16)}
            oracle.kv_write_fp4(pool, [0, 1], range(len(x)), x.view(torch.int16).numpy().view(np.uint16))
            rowsv = oracle.kv_rows_fp4(pool, [0, 1], np.arange(len(x)))
            o = oracle.sink_softmax_attention(oracle.bf16_decode(q[i].cpu().view(torch.int16).numpy().view(np.uint16)), rowsv,
                                              np.zeros(H), 512 ** -0.5)
            # P (numerator and denominator) and the output are rounded to BF16, 2^-8 of a value each
            assert np.abs(out[i].double().cpu().numpy() - o).max() <= 3 * 2.0 ** -8 * np.abs(rowsv).max()
        return out

    a = attend(c.descs, c.d_table, [0, 1, 2, 3])
    L.dsv4sa_cache_release(c.cache, i32([0, 2]))
    table = c.d_table.cpu().numpy()
    np.testing.assert_array_equal(c.d_use.cpu().numpy(), oracle.use_counts(table, P))
    b = attend(c.descs, c.d_table, [1, 3])
    small = Cache(L, (L.POOL_KV_FP4, L.POOL_IDXK_FP4), 5, rows, stride, seed=2)
    new_id, n_used = torch.empty(P, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    L.dsv4sa_cache_compact(c.cache, small.cache, new_id, n_used)
    assert int(n_used) == 2                                # page 20, shared, and the second page of row 1
    assert torch.equal(attend(small.descs, small.d_table, [1, 3]), b)
    L.dsv4sa_cache_compact(c.cache, c.cache, new_id, n_used)
    assert torch.equal(attend(c.descs, c.d_table, [1, 3]), b)
    assert a.shape[0] == 4
