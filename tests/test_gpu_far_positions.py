"""The rotation table at far positions against angles of 90 decimal digits.

A frequency is the nearest multiple of 2^-64 turn, so position n is off by n 2^-65 turn, below n
2^-62.  The remainder, at most pi / 4, is four roundings in fp32 (its two words, the constant, the
product): 4 * 2^-24 * pi / 4 < 2^-22; sine and cosine are a cut series (2^-28) and roundings of
at most 2^-24 and of the inner terms: below 2^-23.  Together 3 * 2^-23 + n 2^-62.  A frequency
held in fp64 would add n 2^-53: 2^-17 at 2^36, where the bound is 2^-21.
"""
import math
from decimal import Decimal as D
from decimal import getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PI = D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def frequencies(pairs, base, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    w = [D(base) ** (D(-i) / pairs) for i in range(pairs)]
    if original_len == 0:
        return [x / D(factor) for x in w]
    border = [pairs * math.log(original_len / (2 * math.pi * b)) / math.log(base) for b in (beta_fast, beta_slow)]
    lo, hi = max(math.floor(border[0]), 0), min(math.ceil(border[1]), 2 * pairs - 1)
    ramp = [D(min(max(i - lo, 0), hi - lo)) / (hi - lo) for i in range(pairs)]
    return [x * (1 - r) + x / D(factor) * r for x, r in zip(w, ramp)]


@pytest.mark.parametrize("first", [0, 2 ** 20, 2 ** 31 - 4, 2 ** 36 + 1, 2 ** 40 - 1])
@pytest.mark.parametrize("kw", [dict(pairs=32, base=160000.0, factor=16.0, original_len=65536), dict(pairs=1, base=10000.0),
                                dict(pairs=48, base=1e6, factor=3.0), dict(pairs=256, base=1.01)])
def test_angles(L, kw, first):
    getcontext().prec = 90
    rows, pairs = 5, kw["pairs"]
    cs = torch.empty(rows, pairs, 2, device="cuda")
    L.dsv4sa_rope_table(cs, first=first, **{k: v for k, v in kw.items() if k != "pairs"})
    assert L.dsv4sa_check_errors() == (0, 0)
    turn = 2 * PI
    ang = np.array([[float((first + r) * w % turn) for w in frequencies(**kw)] for r in range(rows)])
    got = cs.double().cpu().numpy()
    bound = 3 * 2.0 ** -23 + first * 2.0 ** -62
    assert np.abs(got[..., 0] - np.cos(ang)).max() <= bound
    assert np.abs(got[..., 1] - np.sin(ang)).max() <= bound
