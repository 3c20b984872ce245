"""The rotation table and rotated heads on the GPU against fp64.

Table.  A frequency is fp64 (a power, a division and the ramp: below 8 * 2^-53 of it), its
phase 64 bits of a turn (2^-64 turn a position), so an angle theta is off by theta * 2^-50 at
most before it is reduced.  Reduced, it is rounded to fp32 as a part of half a turn in
[-1, 1): half a step of 2^-24 there, times pi; sine and cosine are a unit in the last place
(2^-23 of at most 1) off: together below 2 * 2^-23 + theta * 2^-50.

Heads.  The table's fp32 values are exact inputs.  A rotated value is two products and a sum in
fp32 of values that the norm's factor has multiplied (4 roundings at most, 2^-24 each, of
|a| + |b|); the factor is a sum of up to 1024 squares by at most 40 roundings in a row, a
mean, eps and a reciprocal root (2^-24 (40 / 2 + 4)): 2^-18 of the magnitudes covers both.  The
output is rounded once: 2^-8 of it.
"""
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


YARN = dict(base=160000.0, factor=16.0, original_len=65536)


@pytest.mark.parametrize("rows,pairs,first,kw", [
    (1, 1, 0, dict(base=10000.0)), (1, 32, 7, YARN), (3, 256, 0, YARN), (1000, 32, 0, YARN), (777, 32, 2 ** 20 - 3, YARN),
    (257, 20, 12345, dict(base=500.0, factor=4.0)), (64, 7, 2 ** 40, dict(base=10000.0)), (5000, 64, 3, dict(base=1.5)),
    (100, 16, 0, dict(base=10000.0, factor=8.0, original_len=4096, beta_fast=20.0, beta_slow=2.0))])
def test_table(L, rows, pairs, first, kw):
    cs = torch.full((rows + 1, pairs, 2), 7.0, device="cuda")
    L.dsv4sa_rope_table(cs[:rows], first=first, **kw)
    assert L.dsv4sa_check_errors() == (0, 0)
    w = oracle.yarn_freqs(pairs, **kw)
    pos = first + np.arange(rows, dtype=np.float64)
    ang = np.outer(pos, w)
    got = cs.cpu().double().numpy()
    bound = 2 * 2.0 ** -23 + ang * 2.0 ** -50
    # of far positions numpy's own product is a rounding off as well (2^-53 of the angle)
    assert (np.abs(got[:rows, :, 0] - np.cos(ang)) <= bound + ang * 2.0 ** -52).all()
    assert (np.abs(got[:rows, :, 1] - np.sin(ang)) <= bound + ang * 2.0 ** -52).all()
    assert (got[rows] == 7.0).all()


def test_small_angles_keep_their_relative_precision(L):
    """The slowest pairs of a scaled context turn by 1e-7 a position: sin(x) is x there."""
    cs = torch.empty(16, 32, 2, device="cuda")
    L.dsv4sa_rope_table(cs, **YARN)
    ang = np.outer(np.arange(16, dtype=np.float64), oracle.yarn_freqs(32, **YARN))
    small = (ang < 1e-3) & (ang > 0)
    assert small.sum() > 100
    # the argument's rounding and the sine's: 2^-24 + 2^-23 of it
    rel = np.abs(cs[..., 1].cpu().double().numpy() / np.sin(np.where(small, ang, 1.0)) - 1)[small]
    assert rel.max() <= 2 * 2.0 ** -23


def heads(rng, shape, spread=1.0):
    x = rng.standard_normal(shape).astype(np.float32) * np.exp2(spread * rng.standard_normal(shape[-1])).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


def table_of(L, rows, pairs):
    cs = torch.empty(rows, pairs, 2, device="cuda")
    L.dsv4sa_rope_table(cs, **YARN)
    return cs


def expected(x, cs, pos, off, halves, inverse, eps, w):
    """(value, magnitude behind it) in fp64."""
    x = x.double().cpu().numpy()
    if eps is not None:
        x = oracle.rms_norm(x, 1.0 if w is None else w.double().cpu().numpy(), eps)
    row = cs.double().cpu().numpy()[pos.cpu().numpy()]
    z = (row[..., 0] + 1j * row[..., 1])[:, None, :]
    n = z.shape[-1]
    mag = np.abs(x)
    a = np.arange(n) + off if halves else 2 * np.arange(n) + off
    b = a + n if halves else a + 1
    both = mag[..., a] + mag[..., b]
    mag[..., a], mag[..., b] = both, both
    return oracle.rotate_heads(x, z, off, halves, inverse), mag


def check(got, want, mag):
    got = got.double().cpu().numpy()
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag)
    assert over.max() <= 0, (over.max(), np.argwhere(over > 0)[:4])


CASES = [(1, 1, 512, 64, None), (3, 5, 512, 64, None), (37, 64, 128, 64, None), (7, 3, 64, 64, None), (5, 2, 16, 16, None),
         (9, 7, 1024, 512, None), (4, 3, 520, 48, 8), (2, 128, 40, 16, 16), (300, 2, 192, 64, 0), (33, 1, 768, 256, 512),
         (6, 5, 512, 512, None), (11, 4, 256, 80, 72)]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,H,dim,rd,off", CASES)
def test_heads_match_oracle(L, T, H, dim, rd, off, halves):
    rng = np.random.default_rng(T * 1000 + dim)
    layout = L.ROPE_HALVES if halves else L.ROPE_PAIRS
    cs = table_of(L, 999, rd // 2)
    pos = torch.from_numpy(rng.integers(0, 999, T).astype(np.int32)).cuda()
    at = dim - rd if off is None else off
    w = torch.from_numpy(rng.uniform(0.5, 1.5, dim).astype(np.float32)).cuda()
    for inverse, eps, weight in ((False, None, None), (True, None, None), (False, 1e-6, None), (True, 1e-3, w)):
        x = heads(rng, (T, H, dim))
        want, mag = expected(x, cs, pos, at, halves, inverse, eps, weight)
        out = torch.full((T + 1, H, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        keep = x.clone()
        L.dsv4sa_rope(x, cs, pos, out=out[:T], rope_off=off, layout=layout, inverse=inverse, eps=eps, norm_w=weight)
        check(out[:T], want, mag)
        assert (out[T] == 7).all() and torch.equal(x, keep)
        L.dsv4sa_rope(x, cs, pos, rope_off=off, layout=layout, inverse=inverse, eps=eps, norm_w=weight)   # in place
        assert torch.equal(x.view(torch.int16), out[:T].view(torch.int16))
    assert L.dsv4sa_check_errors() == (0, 0)


@pytest.mark.parametrize("halves", [False, True])
def test_strides(L, halves):
    """Heads before tokens, gaps between rows, a token for all heads, one output inside another tensor."""
    rng = np.random.default_rng(8)
    layout = L.ROPE_HALVES if halves else L.ROPE_PAIRS
    cs = table_of(L, 50, 32)
    T, H = 13, 6
    pos = torch.from_numpy(rng.integers(0, 50, T).astype(np.int32)).cuda()
    base = heads(rng, (H, T, 200))
    x = base.transpose(0, 1)[:, :, 8:136]                       # [T, H, 128], offset 16 bytes
    want, mag = expected(x, cs, pos, 64, halves, False, 1e-6, None)
    store = torch.full((T, H + 2, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    out = store[:, 1:H + 1, 8:136]
    L.dsv4sa_rope(x, cs, pos, out=out, layout=layout, eps=1e-6)
    check(out, want, mag)
    store[:, 1:H + 1, 8:136] = 7.0
    assert (store == 7).all()
    shared = heads(rng, (T, 1, 128)).expand(T, H, 128)          # one key for all heads
    want, mag = expected(shared, cs, pos, 64, halves, False, None, None)
    L.dsv4sa_rope(shared, cs, pos, out=out, layout=layout)
    check(out, want, mag)
    before = base.clone()
    want, mag = expected(x, cs, pos, 64, halves, False, None, None)
    L.dsv4sa_rope(x, cs, pos, layout=layout)                    # in place, strided: the rest stays
    check(x, want, mag)
    x[:] = before.transpose(0, 1)[:, :, 8:136]
    assert torch.equal(base.view(torch.int16), before.view(torch.int16))
    assert L.dsv4sa_check_errors() == (0, 0)


def test_position_out_of_the_table(L):
    rng = np.random.default_rng(9)
    cs = table_of(L, 10, 32)
    pos = torch.tensor([3, 10, -1, 9], dtype=torch.int32, device="cuda")
    x = heads(rng, (4, 3, 128))
    want, mag = expected(x, cs, torch.tensor([3, 0, 0, 9]), 64, False, False, 1e-6, None)
    plain = oracle.rms_norm(x.double().cpu().numpy(), 1.0, 1e-6)
    want[1:3], mag[1:3] = plain[1:3], np.abs(plain[1:3])
    out = torch.empty_like(x)
    L.dsv4sa_rope(x, cs, pos, out=out, eps=1e-6)
    assert L.dsv4sa_check_errors() == (5, 1)
    check(out, want, mag)
    keep = x.clone()
    L.dsv4sa_rope(x, cs, pos)
    assert L.dsv4sa_check_errors() == (5, 1)
    assert torch.equal(x[1:3], keep[1:3]) and not torch.equal(x[0], keep[0])


def test_rotating_there_and_back(L):
    """The inverse is the gradient of the rotation: grad_x = rotate back(grad_out), here by differences."""
    rng = np.random.default_rng(10)
    cs = table_of(L, 40, 32)
    pos = torch.from_numpy(rng.integers(0, 40, 6).astype(np.int32)).cuda()
    g = heads(rng, (6, 2, 128), 0.0)
    back = torch.empty_like(g)
    L.dsv4sa_rope(g, cs, pos, out=back, inverse=True)
    for d in (0, 64, 65, 100, 127):
        # a unit step of x[.., d]: BF16 holds it, the rotation is linear
        e = torch.zeros_like(g)
        e[..., d] = 1.0
        r = torch.empty_like(g)
        L.dsv4sa_rope(e, cs, pos, out=r)
        diff = (r.double() * g.double()).sum(-1)
        # the two results and r are BF16: 2^-8 of each product
        bound = 2.0 ** -7 * ((r.double() * g.double()).abs().sum(-1) + back[..., d].double().abs()) + 1e-6
        assert ((diff - back[..., d].double()).abs() <= bound).all()


def test_graph_stream_and_empty(L):
    rng = np.random.default_rng(11)
    cs = table_of(L, 100, 32)
    pos = torch.from_numpy(rng.integers(0, 100, 50).astype(np.int32)).cuda()
    x = heads(rng, (50, 4, 512))
    ref, out = torch.empty_like(x), torch.zeros_like(x)
    L.dsv4sa_rope(x, cs, pos, out=ref, eps=1e-6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    table = torch.zeros_like(cs)
    with torch.cuda.graph(g, stream=s):
        L.dsv4sa_rope_table(table, **YARN)
        L.dsv4sa_rope(x, table, pos, out=out, eps=1e-6)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    L.dsv4sa_rope(x, cs, pos, out=out, eps=1e-6, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    L.dsv4sa_rope(x[:0], cs, pos, out=out[:0])
    L.dsv4sa_rope_table(cs[:0])
    assert L.dsv4sa_check_errors() == (0, 0)


def test_many_rows(L):
    """More rows than run at once; far token strides (offsets past 2^31 bytes)."""
    rng = np.random.default_rng(12)
    cs = table_of(L, 4096, 32)
    T, H = 20011, 8
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 4096
    x = torch.randn(T, H, 512, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    L.dsv4sa_rope(x, cs, pos, out=out, eps=1e-6)
    at = rng.integers(0, T, 50)
    want, mag = expected(x[at], cs, pos[at], 448, False, False, 1e-6, None)
    check(out[at], want, mag)
    wide = torch.zeros(5, 300_000_000, dtype=torch.bfloat16, device="cuda")     # 600 MB between tokens
    view = wide[:, :1024].view(5, 2, 512)
    view.copy_(x[:5, :2])
    L.dsv4sa_rope(view, cs, pos, eps=1e-6)
    assert torch.equal(view.contiguous().view(torch.int16), out[:5, :2].contiguous().view(torch.int16))
    assert L.dsv4sa_check_errors() == (0, 0)
