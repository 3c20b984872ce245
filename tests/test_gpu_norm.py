"""RMSNorm with the residual's addition and E4M3 output (dsv4sa_rmsnorm_quant) against
the oracle in fp64.

Bounds (a BF16 rounding moves a value by at most half a step of its 8 significant
bits, 2^-8 of it).  s: BF16 of a sum of two BF16 values in fp32 (exact or one fp32
rounding), so |err| <= (2^-8 + 2^-23) |s|.  y in fp32: s carries 2^-24; the sum of squares is
dim terms in a tree of depth <= 32 + 9 + 16 sequential additions, relative 2^-24 * 64;
rsqrt, two products and eps: together |y err| <= 2^-24 * 48 |y| =: e_y (half of the
sum's 64, plus 16), and 2^-8 more in BF16.  scale: e_y + 2 * 2^-24.  A code is the
nearest E4M3 value of z = y / scale moved by at most 2^-24 * 128 of z: half a step
(2^-4 relative for normal values, 2^-10 below 2^-6) plus that.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def make(n, dim, seed, stride=None, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, stride or dim, generator=g) * scale * torch.exp2(2 * torch.randn(stride or dim, generator=g))
    return x.to(torch.bfloat16).cuda()[:, :dim]


def within(err, bound):
    bad = int((np.abs(err) > bound).sum())
    assert bad == 0, f"{bad} of {err.size} off, by up to {np.max(np.abs(err) / np.maximum(bound, 1e-300)):.3g} of the bound"


def check(ref, sum_=None, y=None, codes=None, scale=None):
    if sum_ is not None:
        within(sum_.double().cpu().numpy() - ref["s"], (2.0 ** -8 + 2 * U) * np.abs(ref["s"]))
    if y is not None:
        within(y.double().cpu().numpy() - ref["y"], (2.0 ** -8 + 48 * U) * np.abs(ref["y"]) + 1e-38)
    if codes is not None:
        within(scale.double().cpu().numpy() - ref["scale"], 52 * U * ref["scale"])
        z = ref["z"]
        half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -9)))) * 2.0 ** -4, 2.0 ** -10)
        within(oracle.e4m3_decode(codes.cpu().numpy()) - z, half + 128 * U * np.abs(z))


@pytest.mark.parametrize("n,dim,group", [(1, 64, 64), (5, 128, 64), (1000, 128, 128), (33, 192, 64), (7, 512, 64), (3, 576, 64),
                                         (17, 1024, 128), (2, 1536, 128), (700, 2048, 64), (9, 4096, 128), (400, 7168, 128), (3, 16384, 64),
                                         (2, 8320, 64)])
def test_norm_matches_fp64(L, n, dim, group):
    x, r = make(n, dim, n + dim), make(n, dim, n + dim + 1, scale=3.0)
    w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(dim))).cuda()
    for residual in (None, r):
        codes = torch.full((n, dim), 77, dtype=torch.uint8, device="cuda")
        scale = torch.full((n, dim // group), -1.0, device="cuda")
        s, y = torch.empty_like(x), torch.empty_like(x)
        L.dsv4sa_rmsnorm_quant(x, w, codes, scale, group=group, residual=residual, residual_out=s, y=y, eps=1e-5)
        ref = oracle.rms_norm_quant(bits(x), None if residual is None else bits(residual), w.cpu().numpy(), 1e-5, group)
        check(ref, s, y, codes, scale)
        if residual is None:
            assert torch.equal(s, x)
        # each output alone gives the same bits
        c2, s2, y2, t2 = torch.empty_like(codes), torch.empty_like(scale), torch.empty_like(x), torch.empty_like(x)
        L.dsv4sa_rmsnorm_quant(x, w, c2, s2, group=group, residual=residual, eps=1e-5)
        L.dsv4sa_rmsnorm_quant(x, w, group=group, residual=residual, y=y2, eps=1e-5)
        L.dsv4sa_rmsnorm_quant(x, w, group=group, residual=residual, residual_out=t2, eps=1e-5)
        assert torch.equal(codes, c2) and torch.equal(scale, s2) and torch.equal(y, y2) and torch.equal(s, t2)
    assert L.dsv4sa_check_errors() == (0, 0)


def test_strided_rows_and_in_place_residual(L):
    n, dim = 300, 640
    x, r = make(n, dim, 1, stride=1000), make(n, dim, 2, stride=648)
    w = torch.ones(dim, device="cuda")
    codes, scale = torch.empty(n, dim, dtype=torch.uint8, device="cuda"), torch.empty(n, 10, device="cuda")
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale, group=64, residual=r)
    c2, s2, stream = torch.empty_like(codes), torch.empty_like(scale), r.contiguous()
    xc = x.contiguous()
    L.dsv4sa_rmsnorm_quant(xc, w, c2, s2, group=64, residual=stream, residual_out=stream)   # the residual stream in place
    assert torch.equal(codes, c2) and torch.equal(scale, s2)
    assert torch.equal(stream, (x.float() + r.float()).to(torch.bfloat16))
    L.dsv4sa_rmsnorm_quant(xc, w, c2, s2, group=64, residual=r, residual_out=xc)            # into x itself
    assert torch.equal(codes, c2) and torch.equal(xc, stream)


def test_zero_rows_and_floor(L):
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    x[1, :64] = 1.0
    w = torch.ones(256, device="cuda")
    codes, scale, y = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(4, 4, device="cuda"), torch.empty_like(x)
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale, group=64, y=y, eps=1e-6)
    floor = np.float32(1e-4) * np.float32(1 / 448)
    assert (codes[0] == 0).all() and (y[0] == 0).all() and (scale[0].cpu().numpy() == floor).all()
    assert (codes[1, :64] == 0x7E).all() and (codes[1, 64:] == 0).all() and abs(float(y[1, 0]) - 2.0) < 2 ** -7


def test_feeds_the_indexer(L):
    """The codes and scales of [T * Hi, 128] rows are the indexer's q_fp8 and q_scale."""
    rng = np.random.default_rng(0)
    T, Hi, N = 3, 16, 200
    key_codes, key_scale = rng.integers(0, 0x70, (5, 64, 128)).astype(np.uint8), rng.uniform(0.1, 1, (5, 64, 2)).astype(np.float32)
    buf, keys = L.pack_key_pool(key_codes, key_scale)
    pt = torch.tensor([[3, 1, 4, 0]], dtype=torch.int32, device="cuda")
    x = make(T * Hi, 128, 4)
    w = torch.ones(128, device="cuda")
    q, qs = torch.empty(T * Hi, 128, dtype=torch.uint8, device="cuda"), torch.empty(T * Hi, 2, device="cuda")
    L.dsv4sa_rmsnorm_quant(x, w, q, qs, group=64)
    wts = torch.rand(T, Hi, device="cuda")
    logits = torch.empty(T, N, device="cuda")
    seq, nv = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.full((T,), N, dtype=torch.int32, device="cuda")
    L.dsv4sa_indexer_logits(keys, pt, seq, nv, q.view(T, Hi, 128), qs.view(T, Hi, 2), wts, N, logits)
    assert L.dsv4sa_check_errors() == (0, 0)
    for t in range(T):
        ref = oracle.indexer_logits_row(q.view(T, Hi, 128)[t].cpu().numpy(), qs.view(T, Hi, 2)[t].cpu().numpy(), wts[t].cpu().numpy(),
                                        {"codes": key_codes, "scale": key_scale}, pt[0].cpu().numpy(), N)
        qd = np.abs(oracle.index_query(q.view(T, Hi, 128)[t].cpu().numpy(), qs.view(T, Hi, 2)[t].cpu().numpy()))
        kd = np.abs(oracle.index_keys({"codes": key_codes, "scale": key_scale}, pt[0].cpu().numpy(), np.arange(N)))
        bound = 2e-5 * ((kd @ qd.T) @ np.abs(wts[t].cpu().numpy().astype(np.float64)))   # as in tests/parity.py
        assert (np.abs(logits[t].cpu().numpy() - ref) <= bound + 1e-30).all()


def test_graph_replay_and_side_stream(L):
    x, r = make(64, 4096, 7), make(64, 4096, 8)
    w = torch.ones(4096, device="cuda")
    codes, scale = torch.empty(64, 4096, dtype=torch.uint8, device="cuda"), torch.empty(64, 32, device="cuda")
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale, residual=r)
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.dsv4sa_rmsnorm_quant(x, w, c2, s2, residual=r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(codes, c2) and torch.equal(scale, s2)
