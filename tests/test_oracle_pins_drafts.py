"""Pins of the oracle's rotary tables, appended rows and trees of drafted tokens: hand-worked
values, library routines and invariants, none of them the oracle's own code."""
import math

import numpy as np
import pytest
import torch

import oracle


def test_plain_frequencies_are_the_ones_of_the_output_rotation():
    np.testing.assert_allclose(oracle.yarn_freqs(32, 10000.0), oracle.base_freqs(10000.0), rtol=1e-15)


def test_interpolation_divides_every_frequency():
    np.testing.assert_allclose(oracle.yarn_freqs(16, 500.0, 4.0) * 4, oracle.yarn_freqs(16, 500.0), rtol=1e-15)


@pytest.mark.parametrize("pairs,base,factor,length", [(32, 160000.0, 16.0, 65536), (64, 10000.0, 40.0, 4096), (8, 1000.0, 2.0, 512)])
def test_yarn_keeps_fast_pairs_and_divides_slow_ones(pairs, base, factor, length):
    w, y = oracle.yarn_freqs(pairs, base), oracle.yarn_freqs(pairs, base, factor, length)
    turns = length * w / (2 * math.pi)
    ratio = w / y
    assert ratio.min() >= 1 - 1e-12 and ratio.max() <= factor * (1 + 1e-12)
    assert (np.diff(ratio) >= -1e-12).all()                       # slower pairs are scaled more
    # a pair next to a border may lie on the ramp: whole pair numbers
    i = np.arange(pairs)
    fast = i <= np.floor(pairs * np.log(length / (2 * math.pi * 32)) / np.log(base))
    slow = i >= np.ceil(pairs * np.log(length / (2 * math.pi)) / np.log(base))
    assert (turns[fast] >= 32 * (1 - 1e-9)).all() and (turns[slow] <= 1 + 1e-9).all()
    np.testing.assert_allclose(ratio[fast], 1.0, rtol=1e-12)
    np.testing.assert_allclose(ratio[slow], factor, rtol=1e-12)


def test_yarn_ramp_by_hand():
    # 4 pairs, base 16: w = 1, 1/2, 1/4, 1/8.  Borders at 4 log_16(100 / (2 pi beta)): beta 10 -> 0.67, beta 1 -> 3.99
    w = oracle.yarn_freqs(4, 16.0, 2.0, 100, 10.0, 1.0)
    ramp = np.array([0, 0.25, 0.5, 0.75])                          # (i - 0) / (4 - 0)
    np.testing.assert_allclose(w, np.array([1, 0.5, 0.25, 0.125]) * (1 - ramp / 2), rtol=1e-12)


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_is_the_matrix_of_its_angles(halves):
    rng = np.random.default_rng(3)
    x, ang = rng.standard_normal((5, 40)), rng.uniform(-7, 7, 8)
    got = oracle.rotate_heads(x, np.exp(1j * ang), 16, halves)
    m = np.eye(40)
    for i in range(8):
        a, b = (16 + i, 24 + i) if halves else (16 + 2 * i, 17 + 2 * i)
        m[a, a] = m[b, b] = math.cos(ang[i])
        m[a, b], m[b, a] = -math.sin(ang[i]), math.sin(ang[i])
    np.testing.assert_allclose(got, x @ m.T, atol=1e-12)
    np.testing.assert_allclose(oracle.rotate_heads(got, np.exp(1j * ang), 16, halves, inverse=True), x, atol=1e-12)


def test_inverse_rotation_is_the_gradient():
    # d(sum(g * rotate(x))) / dx by differences
    rng = np.random.default_rng(4)
    x, g, row = rng.standard_normal(32), rng.standard_normal(32), np.exp(1j * rng.uniform(-3, 3, 16))
    grad = oracle.rotate_heads(g, row, 0, True, inverse=True)
    h = 1e-6
    for d in range(32):
        e = np.zeros(32)
        e[d] = h
        diff = ((oracle.rotate_heads(x + e, row, 0, True) - oracle.rotate_heads(x - e, row, 0, True)) * g).sum() / (2 * h)
        assert abs(diff - grad[d]) < 1e-8


def test_appended_row_against_torch():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal(512).astype(np.float32)).to(torch.bfloat16)
    w = rng.uniform(0.5, 1.5, 512)
    row = np.exp(1j * rng.uniform(-3, 3, 32))
    y = torch.nn.functional.rms_norm(x.double(), (512,), torch.from_numpy(w), 1e-3)
    z = torch.view_as_complex(y[448:].reshape(32, 2)) * torch.from_numpy(row)
    want = torch.cat((y[:448], torch.view_as_real(z).reshape(-1))).numpy()
    np.testing.assert_allclose(oracle.append_row(x.view(torch.int16).numpy().view(np.uint16), row, w, 1e-3), want, atol=1e-12)


def test_masks_and_window_by_hand():
    #      0
    #     / \
    #    1   2      node 3 follows 2; node 4 is a second root
    masks = oracle.tree_masks([-1, 0, 0, 2, -1])
    assert masks == [0b1, 0b11, 0b101, 0b1101, 0b10000]
    # 5 committed tokens, a window of 4 over a ring of 3, drafted rows from slot 10: node 3 stands at 5 + 2
    win, drafts = oracle.tree_window(7, 5, 4, 3, masks[3], 5, 10)
    assert win.tolist() == [1, -1, -1, -1] and drafts.tolist() == [10, -1, 12, 13, -1]
    # position 4 of a context of 5: all committed, no drafted rows kept
    win, drafts = oracle.tree_window(4, 5, 4, 0, 1, 1, -1)
    assert win.tolist() == [1, 2, 3, 4] and drafts.tolist() == [-1]


def test_a_chain_is_causal_attention():
    # the nodes of a chain after ctx tokens: torch's causal attention over the same rows
    rng = np.random.default_rng(6)
    ctx, n, H = 7, 4, 3
    rows, q = rng.standard_normal((ctx + n, 512)), rng.standard_normal((n, H, 512))
    masks = oracle.tree_masks([-1, 0, 1, 2])
    kv = torch.from_numpy(rows).expand(H, -1, -1)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), kv, kv, torch.ones(n, ctx + n, dtype=torch.bool).tril(ctx), scale=0.1).transpose(0, 1)
    for t in range(n):
        win, drafts = oracle.tree_window(ctx + t, ctx, 64, 0, masks[t], n, ctx)
        seen = [e for e in list(win) + list(drafts) if e >= 0]
        assert seen == list(range(ctx + t + 1))
        got = oracle.sink_softmax_attention(q[t], rows[seen], np.full(H, -np.inf), 0.1)
        np.testing.assert_allclose(got, want[t].numpy(), atol=1e-12)


def test_lse_with_and_without_rows():
    rng = np.random.default_rng(7)
    q, rows, sink = rng.standard_normal((2, 512)), rng.standard_normal((5, 512)), np.array([0.3, -np.inf])
    a = torch.from_numpy(np.concatenate([0.2 * q @ rows.T, sink[:, None]], 1))
    np.testing.assert_allclose(oracle.attend_lse(q, rows, sink, 0.2), torch.logsumexp(a, 1).numpy(), rtol=1e-12)
    none = oracle.attend_lse(q, np.zeros((0, 512)), sink, 0.2)
    assert none[0] == 0.3 and np.isneginf(none[1])
