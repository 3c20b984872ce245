"""The FP4 KV cache on the GPU: rows written and read back (byte for byte and value
for value against the oracle: quantisation is decided in fp32 on both sides and
dequantisation is exact in BF16), and sparse attention over it against fp64.

Tolerance of the attention.  The rows are exact.  P is rounded to BF16 (half a
step of its 8 significant bits: 2^-8 of each probability) for the numerator, which
so moves by at most 2^-8 of sum_j p_j |kv_jd|, and the output is rounded to BF16
(2^-8 of the value); the sum of the probabilities is fp32.  The scores are fp32 sums of 512 exact
products: error at most 512 * 2^-24 * scale * sum_d |q_d kv_jd| =: eps_s per
score, which moves p_j by a factor e^eps_s.  Together, per element,
  |err| <= (2^-8 + 2 eps_s + 2^-16) * A + 2^-8 |o|,  A = sum_j p_j |kv_jd| / Z
with 2^-16 for the fp32 accumulation over up to 2048 rows, the exponentials and
the log-sum-exp merge.  Below fp32's normal range a probability (against a max at
most the row's) is flushed to zero: 2^-126 max |kv| for each row more, absolute,
as Z >= 1 against the row's max.  |lse err| <= eps_s + 2^-16 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module")
def L():
    import os
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


def bits_of(x):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def bf16_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def unpack(L, buf, P):
    d = L.dsv4sa_pool_desc_init(L.POOL_KV_FP4, 1 << 20, P)
    host = buf.cpu().numpy().reshape(P, d.page_stride)
    packed = host[:, :64 * 224].reshape(P, 64, 224)
    codes = np.empty((P, 64, 448), np.uint8)
    codes[..., 0::2], codes[..., 1::2] = packed & 15, packed >> 4
    rope = np.ascontiguousarray(host[:, d.rope_off:d.rope_off + 64 * 128]).view(np.uint16).reshape(P, 64, 64)
    sc = host[:, d.scale_off:].reshape(P, 64, 16)
    return {"nope_codes": codes, "nope_e8m0": sc[..., :14].copy(), "rope_bits": rope.copy()}, sc[..., 14:]


def random_pool(rng, P, lo=120, hi=131):
    return {"nope_codes": rng.integers(0, 16, (P, 64, 448)).astype(np.uint8),
            "nope_e8m0": rng.integers(lo, hi, (P, 64, 14)).astype(np.uint8),
            "rope_bits": bits_of(rng.standard_normal((P, 64, 64)))}


def special_rows(rng, n):
    """Blocks of every magnitude, zeros, negative zeros, E2M1 ties, the largest and
    smallest BF16 values, infinities and NaN."""
    x = rng.standard_normal((n, 512)).astype(np.float32) * np.exp2(rng.integers(-30, 30, (n, 16)).astype(np.float32)).repeat(32, 1)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0], np.float32)
    rows = [lambda r: r.__setitem__(slice(None), 0.0),
            lambda r: r.__setitem__(slice(None, None, 3), -0.0),
            lambda r: r.__setitem__(slice(0, 448), np.tile(ties, 28)),
            lambda r: r.__setitem__(slice(0, 448), np.tile(ties, 28) * np.float32(2.0 ** 20)),
            lambda r: r.__setitem__(slice(32, 64), 3e38),
            lambda r: r.__setitem__(slice(64, 96), 1e-40),
            lambda r: r.__setitem__(100, np.inf),
            lambda r: r.__setitem__(447, np.nan),
            lambda r: r.__setitem__(500, np.nan)]
    for i, f in enumerate(rows[:n]):
        f(x[i])
    return bits_of(x)


@pytest.mark.parametrize("n", [1, 3, 37, 700])
def test_write_and_read_match_oracle(L, n):
    rng = np.random.default_rng(40 + n)
    P, B = 30, 3
    pool = random_pool(rng, P)
    pt = rng.permutation(P)[:B * 9].reshape(B, 9).astype(np.int32)
    pairs = rng.permutation(B * 576)[:n]
    seq, ent = (pairs // 576).astype(np.int32), (pairs % 576).astype(np.int32)
    bits = special_rows(rng, n)
    buf, desc = L.pack_kv_pool_fp4(pool["nope_codes"], pool["nope_e8m0"], pool["rope_bits"])
    L.dsv4sa_cache_write(desc, dev(pt), dev(seq), dev(ent), bf16_dev(bits))
    back = torch.full((n, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    L.dsv4sa_cache_read(desc, dev(pt), dev(seq), dev(ent), back)
    assert L.dsv4sa_check_errors() == (0, 0)
    ref = {k: v.copy() for k, v in pool.items()}
    for r in range(n):
        oracle.kv_write_fp4(ref, pt[seq[r]], [ent[r]], bits[r:r + 1])
    got, pad = unpack(L, buf, P)
    for k in ref:
        bad = np.argwhere(got[k] != ref[k])
        assert bad.size == 0, (k, bad[:4])
    assert (pad == 0).all()                      # the padding of the scale rows is never written
    want = np.stack([oracle.kv_rows_fp4(ref, pt[seq[r]], [ent[r]])[0] for r in range(n)])
    # BF16 holds every value (2 significant bits) but 4 * 2^126 = 2^128, past its range: an infinity
    assert (np.abs(want[np.isfinite(want)]) <= 2.0 ** 128).all()
    want = np.where(np.abs(want) == 2.0 ** 128, np.copysign(np.inf, want), want)
    np.testing.assert_array_equal(back.double().cpu().numpy(), want)


def test_read_of_missing_rows_and_fp8_pools(L):
    rng = np.random.default_rng(9)
    P = 5
    pool = random_pool(rng, P)
    buf, desc = L.pack_kv_pool_fp4(pool["nope_codes"], pool["nope_e8m0"], pool["rope_bits"])
    pt = np.array([[4, 2, 0], [1, 9, -3]], np.int32)          # row 1: two pages out of range
    seq = np.array([0, 0, 0, 1, 1, 1, -1], np.int32)
    ent = np.array([191, -1, 192, 5, 64, 128, 3], np.int32)
    out = torch.full((7, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    L.dsv4sa_cache_read(desc, dev(pt), dev(seq[:2]), dev(ent[:2]), out[:2])
    assert L.dsv4sa_check_errors() == (0, 0)                  # -1 is no error
    L.dsv4sa_cache_read(desc, dev(pt), dev(seq), dev(ent), out)
    assert L.dsv4sa_check_errors() == (5, 1)
    want = np.zeros((7, 512))
    want[0] = oracle.kv_rows_fp4(pool, pt[0], [191])[0]
    want[3] = oracle.kv_rows_fp4(pool, pt[1], [5])[0]
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)
    # FP8 pools: e4m3(code) * scale, rounded to BF16 once
    codes = rng.integers(0, 0x7F, (P, 64, 448)).astype(np.uint8)
    scale = rng.uniform(0.01, 2, (P, 64, 7)).astype(np.float32)
    buf8, d8 = L.pack_kv_pool(codes, scale, pool["rope_bits"])
    ent = np.arange(0, 190, 7, dtype=np.int32)
    out = torch.empty(len(ent), 512, dtype=torch.bfloat16, device="cuda")
    L.dsv4sa_cache_read(d8, dev(pt), dev(np.zeros(len(ent), np.int32)), dev(ent), out)
    assert L.dsv4sa_check_errors() == (0, 0)
    rows = oracle.kv_rows({"nope_codes": codes, "nope_scale": scale, "rope_bits": pool["rope_bits"]}, pt[0], ent)
    fp32 = torch.from_numpy(rows).float()                      # the product in fp32 (one rounding), then BF16
    assert torch.equal(out.cpu(), fp32.to(torch.bfloat16))


def attention_reference(q_bits, sink, rows):
    """o [H, 512], lse [H], and the bounds of the docstring for both."""
    q = oracle.bf16_decode(q_bits)
    o = oracle.sink_softmax_attention(q, rows, sink, SCALE)
    if rows.shape[0] == 0:
        return o, sink.astype(np.float64), np.zeros_like(o), 2.0 ** -22 * np.abs(sink)
    a = SCALE * (q @ rows.T)
    M = np.maximum(a.max(1), sink)
    p = np.exp(a - M[:, None])
    Z = p.sum(1) + np.exp(sink - M)
    A = (p @ np.abs(rows)) / Z[:, None]
    eps_s = (512 * 2.0 ** -24 * SCALE * (np.abs(q) @ np.abs(rows).T)).max(1)
    tol = (2.0 ** -8 + 2 * eps_s[:, None] + 2.0 ** -16) * A + 2.0 ** -8 * np.abs(o)
    tol += rows.shape[0] * 2.0 ** -126 * np.abs(rows).max()
    return o, M + np.log(Z), tol, eps_s + 2.0 ** -16 + 2.0 ** -22 * np.abs(M + np.log(Z))


class Case:
    """T queries over B sequences of `entries` compressed entries in FP4 pools."""

    def __init__(self, L, T, H, kc, kw, seed, B=2, entries=1500, ring=0, q_scale=1.0, empty=(), pool_lo=124, pool_hi=128):
        rng = np.random.default_rng(seed)
        per = -(-entries // 64)
        self.comp = random_pool(rng, B * per + 1, pool_lo, pool_hi)
        self.comp_pt = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        wper = max(1, -(-(ring or 400) // 64))
        self.win = random_pool(rng, B * wper + 1, pool_lo, pool_hi)
        self.win_pt = rng.permutation(B * wper + 1)[:B * wper].reshape(B, wper).astype(np.int32)
        self.q_bits = bits_of(q_scale * rng.standard_normal((T, H, 512)))
        self.sink = rng.standard_normal(H).astype(np.float32)
        self.seq = rng.integers(0, B, T).astype(np.int32)
        self.idx = np.full((T, kc), -1, np.int32)
        for t in range(T):
            if t in empty:
                continue
            n = rng.integers(0, kc + 1) if t % 3 == 1 else kc
            picks = rng.integers(0, entries, n)                 # duplicates count twice
            where = np.sort(rng.permutation(kc)[:n])            # -1 anywhere between them
            self.idx[t, where] = picks
        self.pos = rng.integers(0, ring * 5 if ring else 399, T).astype(np.int32)
        for t in empty:
            self.pos[t] = -1
        self.kw, self.ring, self.T, self.H, self.kc = kw, ring, T, H, kc
        self.comp_buf, self.comp_d = L.pack_kv_pool_fp4(self.comp["nope_codes"], self.comp["nope_e8m0"], self.comp["rope_bits"])
        self.win_buf, self.win_d = L.pack_kv_pool_fp4(self.win["nope_codes"], self.win["nope_e8m0"], self.win["rope_bits"])
        self.d = dict(q=bf16_dev(self.q_bits), sink=dev(self.sink), seq=dev(self.seq), comp_pt=dev(self.comp_pt),
                      win_pt=dev(self.win_pt), idx=dev(self.idx), pos=dev(self.pos))

    def window(self, t):
        return oracle.window_indices(int(self.pos[t]), self.kw, self.ring) if self.kw else np.zeros(0, np.int64)

    def run(self, L, fn, explicit=False, **kw):
        out = torch.full((self.T, self.H, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.H), 9.0, device="cuda")
        d = self.d
        if explicit and self.kw:
            iw = dev(np.stack([self.window(t) for t in range(self.T)]).astype(np.int32))
            win = dict(win_pos=None, kw=None)
        else:
            iw, win = None, dict(win_pos=d["pos"], kw=self.kw, win_ring=self.ring)
        fn(d["q"], d["sink"], d["seq"], self.comp_d, d["comp_pt"], d["idx"] if self.kc else None, self.win_d, d["win_pt"], iw,
           out, SCALE, lse=lse, **win, **kw)
        return out, lse

    def check(self, out, lse, rows=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for t in range(self.T) if rows is None else rows:
            s = self.seq[t]
            kv = oracle.gather_rows_fp4(self.idx[t] if self.kc else None, self.comp, self.comp_pt[s], self.window(t), self.win, self.win_pt[s])
            o, l, tol, ltol = attention_reference(self.q_bits[t], self.sink, kv)
            err = np.abs(out[t] - o) - tol
            worst, finite = float(err.max()), bool(np.isfinite(out[t]).all())
            assert finite and worst <= 0, (t, kv.shape, worst, np.abs(out[t] - o).max())
            assert (np.abs(lse[t] - l) <= ltol).all(), (t, np.abs(lse[t] - l).max())


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("T,H,kc,kw,ring", [(1, 16, 512, 128, 128), (1, 64, 512, 128, 128), (3, 1, 100, 0, 0), (2, 7, 1, 1, 64),
                                            (5, 64, 129, 127, 128), (4, 33, 512, 16, 64), (40, 64, 512, 128, 128), (3, 128, 640, 130, 192),
                                            (2, 16, 2048, 1024, 1024), (9, 100, 0, 128, 128), (160, 8, 200, 128, 128), (2, 48, 77, 300, 0)])
def test_attention_matches_fp64(L, mode, T, H, kc, kw, ring):
    c = Case(L, T, H, kc, kw, seed=T * 1000 + H + kc, ring=ring, empty=(0,) if T in (5, 40, 160) else (),
             entries=3000 if kc > 1500 else 1500)
    fn = L.dsv4sa_sparse_attn_decode if mode == "decode" else L.dsv4sa_sparse_attn_prefill
    out, lse = c.run(L, fn)
    assert L.dsv4sa_check_errors() == (0, 0)
    c.check(out, lse)
    again, lse2 = c.run(L, fn, explicit=True)                 # the window list given; the same bits
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_sharp_scores_and_wide_scales(L):
    """Scores far apart (the running max moves from chunk to chunk) and block scales from 2^-40 to 2^20."""
    c = Case(L, 6, 64, 600, 128, seed=5, ring=128, q_scale=8.0, pool_lo=124, pool_hi=131)
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        c.check(*c.run(L, fn))
    c = Case(L, 4, 20, 300, 64, seed=6, ring=64, q_scale=2.0 ** -18, pool_lo=87, pool_hi=148)
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        c.check(*c.run(L, fn))
    assert L.dsv4sa_check_errors() == (0, 0)


def test_no_rows_at_all_and_infinite_sink(L):
    c = Case(L, 3, 24, 40, 16, seed=8, ring=64, empty=(0, 1, 2))
    for sink in (0.5, -np.inf):
        c.d["sink"].fill_(sink)
        for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
            out, lse = c.run(L, fn)
            assert torch.equal(out, torch.zeros_like(out)) and (lse == sink).all()
    c = Case(L, 5, 24, 300, 16, seed=8, ring=64, empty=(1,))
    c.d["sink"].fill_(-np.inf)
    c.sink[:] = -1e9                                           # as good as none
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        out, lse = c.run(L, fn)
        c.check(out, lse, rows=(0, 2, 3, 4))
        assert (out[1] == 0).all() and (lse[1] == -np.inf).all()


def test_many_items_per_cta_and_empty_rows(L):
    """More queries than CTAs, a third of them without any row, several head groups."""
    c = Case(L, 400, 80, 150, 32, seed=12, ring=64, empty=tuple(range(0, 400, 3)))
    out, lse = c.run(L, L.dsv4sa_sparse_attn_prefill)
    assert L.dsv4sa_check_errors() == (0, 0)
    c.check(out, lse, rows=list(range(0, 400, 17)) + [399, 398, 397])
    dec, lse_d = c.run(L, L.dsv4sa_sparse_attn_decode)         # no split fits: the same work
    assert torch.equal(dec, out) and torch.equal(lse, lse_d)


def test_bits_do_not_depend_on_other_rows_and_repeat(L):
    c = Case(L, 32, 64, 512, 128, seed=3, ring=128)
    a, la = c.run(L, L.dsv4sa_sparse_attn_decode)
    b, lb = c.run(L, L.dsv4sa_sparse_attn_decode)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_pages_are_flagged_and_skipped(L):
    c = Case(L, 4, 16, 64, 0, seed=31)
    c.idx[1, 5] = 64 * c.comp_pt.shape[1]                      # past the table
    c.d["idx"] = dev(c.idx)
    out, lse = c.run(L, L.dsv4sa_sparse_attn_prefill)
    assert L.dsv4sa_check_errors() == (5, 1)
    c.idx[1, 5] = -1                                           # attended as if it were not there
    c.check(out, lse)


def test_rotated_output_early_window_graph_and_streams(L):
    c = Case(L, 12, 64, 512, 128, seed=21, ring=128)
    table = oracle.rope_table(oracle.base_freqs(), 700)
    cs = dev(np.stack([table.real, table.imag], -1).astype(np.float32))
    pos = np.arange(12, dtype=np.int32) * 50
    for fn in (L.dsv4sa_sparse_attn_decode, L.dsv4sa_sparse_attn_prefill):
        out, lse = c.run(L, fn)
        rot, lse_r = c.run(L, fn, rope_cs=cs.view(700, 32, 2), rope_pos=dev(pos))
        assert torch.equal(rot[..., :448], out[..., :448]) and torch.equal(lse, lse_r)
        # rotation of the fp32 output, against the rotation of the BF16 one: two BF16 roundings apart
        x, y = out[..., 448::2].double(), out[..., 449::2].double()
        co, si = cs.view(700, 32, 2)[dev(pos).long()].double().unbind(-1)
        want = torch.stack((x * co[:, None] + y * si[:, None], y * co[:, None] - x * si[:, None]), -1).flatten(-2)
        size = torch.stack((torch.hypot(x, y),) * 2, -1).flatten(-2)
        assert ((rot[..., 448:].double() - want).abs() <= 2 * 2.0 ** -8 * size + 1e-30).all()
        early, lse_e = c.run(L, fn, flags=L.ATTN_EARLY_WINDOW)  # the window in chunks of its own: other sums
        c.check(early, lse_e)
        # two graphs and an eager call on three streams at once: no shared state
        graphs, outs = [], []
        for _ in range(2):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(c.run(L, fn))
            graphs.append((g, s))
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager, _ = c.run(L, fn)
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, out) and torch.equal(l, lse)
        assert torch.equal(eager, out)
    assert L.dsv4sa_check_errors() == (0, 0)


def test_topk_and_attention_in_one_call(L):
    c = Case(L, 10, 64, 512, 128, seed=22, ring=128)
    N = c.comp_pt.shape[1] * 64
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(10, N, generator=g, device="cuda")
    n_vis = torch.tensor([N, 1500, 512, 511, 3, 0, -1, N, 700, 513], dtype=torch.int32, device="cuda")
    idx1 = c.d["idx"].clone()
    idx2 = c.d["idx"].clone()
    L.dsv4sa_topk(logits, n_vis, N, 512, idx1)
    c.d["idx"] = idx1
    out1, lse1 = c.run(L, L.dsv4sa_sparse_attn_decode)
    out2, lse2 = torch.empty_like(out1), torch.empty_like(lse1)
    d = c.d
    L.dsv4sa_topk_sparse_attn_decode(logits, n_vis, N, 512, d["q"], d["sink"], d["seq"], c.comp_d, d["comp_pt"], idx2, c.win_d,
                                     d["win_pt"], None, out2, SCALE, lse=lse2, win_pos=d["pos"], kw=128, win_ring=128)
    assert L.dsv4sa_check_errors() == (0, 0)
    assert torch.equal(idx1, idx2) and torch.equal(out1, out2) and torch.equal(lse1, lse2)
    c.idx = idx1.cpu().numpy()
    c.check(out1, lse1)
