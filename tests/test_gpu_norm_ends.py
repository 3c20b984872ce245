"""The norm where 1 / rms is far from one: eps = 0 and subnormal, means of squares below the
smallest normal number, rows of any size that the header allows (squares, and products with a
weight, in the normal range of fp32).

The bounds are those of test_gpu_norm: the 2^64 that a small mean is formed with is exact, so
no rounding is added."""
import os

import numpy as np
import pytest
import torch

import oracle
from test_gpu_norm import bits, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def run(L, x, w, group, eps, residual=None):
    n, dim = x.shape
    codes, scale = torch.full((n, dim), 77, dtype=torch.uint8, device="cuda"), torch.full((n, dim // group), -1.0, device="cuda")
    s, y = torch.empty_like(x), torch.empty_like(x)
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale, group=group, residual=residual, residual_out=s, y=y, eps=eps)
    ref = oracle.rms_norm_quant(bits(x), None if residual is None else bits(residual), w.cpu().numpy(), float(np.float32(eps)), group)
    check(ref, s, y, codes, scale)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scale)          # the codes alone: the same bits
    L.dsv4sa_rmsnorm_quant(x, w, c2, s2, group=group, residual=residual, eps=eps)
    assert torch.equal(codes, c2) and torch.equal(scale, s2)
    return codes, scale, y


def values(n, dim, seed, exponent):
    """Values of 1/4 to 5/4 times 2^exponent, either sign, and zeros (no value below 1/4, so
    that no square is below 2^(2 exponent - 4))."""
    g = torch.Generator().manual_seed(seed)
    return torch.ldexp(torch.randint(-5, 6, (n, dim), generator=g) / 4, torch.tensor(exponent)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("dim,group", [(128, 64), (192, 64), (512, 128), (1024, 128), (2048, 64), (4096, 128), (16384, 64)])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-38, 1e-30])
def test_one_small_value_in_a_row(L, dim, group, eps):
    """Squares of 2^-124 and 2^-126, the mean over the row below the smallest normal number."""
    x = torch.zeros(4, dim, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[1, dim - 1], x[2, 70], x[3, 64:96] = 2.0 ** -62, -2.0 ** -63, 1.5 * 2.0 ** -62, 2.0 ** -60
    w = (1 + 0.3 * torch.rand(dim, generator=torch.Generator().manual_seed(1))).cuda()
    codes, _, y = run(L, x, w, group, eps)
    assert (codes[0, 4:] == 0).all() and (y[0, 4:] == 0).all() and float(y[0, 3]) > 0 > float(y[1, dim - 1])


@pytest.mark.parametrize("dim,group", [(128, 128), (256, 64), (512, 64), (1024, 64), (4096, 64), (7168, 128)])
@pytest.mark.parametrize("exponent", [-61, -50, -21, 21, 50, 54])
@pytest.mark.parametrize("weight", [2.0 ** -45, 1.0, 2.0 ** 60])
def test_rows_of_any_size(L, dim, group, exponent, weight):
    """x w from 2^-106 to 2^114; y = x w / rms is of the weights' size."""
    g = torch.Generator().manual_seed(dim)
    w = (weight * (1 + 0.3 * torch.randn(dim, generator=g))).cuda()
    x = values(5, dim, dim + 1, exponent)
    run(L, x, w, group, 0.0)
    run(L, x, w, group, 0.0, residual=values(5, dim, dim + 2, exponent))


def test_zero_rows(L):
    """With eps > 0, however small, a row of zeros gives zeros."""
    for dim, eps in ((128, 1e-44), (4096, 1e-38), (1024, 1e-30)):
        codes, scale, y = run(L, torch.zeros(3, dim, dtype=torch.bfloat16, device="cuda"), torch.ones(dim, device="cuda"), 64, eps)
        assert (codes == 0).all() and (y == 0).all() and float(scale.max()) == float(np.float32(1e-4) * np.float32(1 / 448))


def test_rows_keep_their_bits_beside_others(L):
    """A row's result does not depend on what the other rows of the call hold."""
    for dim, group in ((128, 64), (4096, 128)):
        w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(3))).cuda()
        x = values(64, dim, 9, 0)
        codes, scale, y = run(L, x, w, group, 0.0)
        x2 = x.clone()
        x2[1::2] = values(32, dim, 10, -58)
        codes2, scale2, y2 = run(L, x2, w, group, 0.0)
        assert torch.equal(codes[::2], codes2[::2]) and torch.equal(scale[::2], scale2[::2]) and torch.equal(y[::2], y2[::2])
