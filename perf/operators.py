"""The library's serving operators around a 4-bit KV cache, as cases to measure.

Four groups of calls, each as a serving program makes them:

* ``cache``  new BF16 KV rows quantised into the FP4 pool, and the same rows read back as the
  values the cache holds (a prefill chunk attends to what later steps will read);
* ``attn``   sparse attention with a sink over selected compressed entries and a raw-token
  window, both in FP4 pools;
* ``beam``, ``compact``  the pages of a cache: rows released and forked again (shared full
  pages, a copy of the last partial one), and the pages in use moved to the front of other pools;
* ``norm``   RMSNorm of a BF16 stream with the residual added, quantised to E4M3 with block scales.

``run`` computes the plain form in elementary torch operations, or, with ``own`` set, makes the
library's calls.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64
NOPE, ROPE, DIM = 448, 64, 512
KINDS = {"kv": 0, "idxk": 1, "idxk_fp4": 2, "kv_fp4": 3}
# bytes per slot of each block of a page, in the order the blocks lie in it
BLOCKS = {"kv": (448, 128, 32), "idxk": (128, 8), "idxk_fp4": (64, 4), "kv_fp4": (224, 128, 16)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SOFTMAX_SCALE = 1.0 / math.sqrt(512.0)


def page_bytes(kind):
    return PAGE * sum(BLOCKS[kind])


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 32 sequences: one new KV row each
        {"name": "cache: decode batch", "op": "cache", "n": 32, "seqs": 32, "entries": 16384, "spread": 2.0},
        # a long prompt's rows at once
        {"name": "cache: long prompt", "op": "cache", "n": 65529, "seqs": 4, "entries": 16384, "spread": 2.0},
        # one query over a short context, where latency is all
        {"name": "attn: one query", "op": "attn", "mode": "decode", "T": 1, "H": 16, "N": 1024, "kc": 512, "kw": 128,
         "fill": "full", "sharp": 1.0},
        # the 64K-token decode batch
        {"name": "attn: decode 64k", "op": "attn", "mode": "decode", "T": 32, "H": 64, "N": 16384, "kc": 512, "kw": 128,
         "fill": "full", "sharp": 1.0},
        # a mixed batch: short and long contexts, some rows with nothing to attend to
        {"name": "attn: ragged batch", "op": "attn", "mode": "decode", "T": 128, "H": 8, "N": 8192, "kc": 1024, "kw": 128,
         "fill": "ragged", "sharp": 2.0},
        # a 4096-token prompt chunk at the end of a 64K context
        {"name": "attn: prefill chunk", "op": "attn", "mode": "prefill", "T": 4096, "H": 64, "N": 16384, "kc": 512,
         "kw": 128, "fill": "full", "sharp": 1.0},
        # a beam of four over one sequence
        {"name": "beam: four of one", "op": "beam", "seqs": 1, "width": 4, "tokens": 5003, "kinds": "kv_fp4,idxk_fp4",
         "slack": 1.5},
        # beams of four over a batch of 64 sequences, FP8 pools
        {"name": "beam: four of 64", "op": "beam", "seqs": 64, "width": 4, "tokens": 16001, "kinds": "kv,idxk",
         "slack": 1.25},
        # the pages in use of a fragmented cache moved to smaller pools
        {"name": "compact: fragmented cache", "op": "compact", "pages": 49151, "used": 0.6, "rows": 96,
         "kinds": "kv_fp4,idxk_fp4"},
        # a decode batch's residual stream, FP8 for the projections
        {"name": "norm: decode batch", "op": "norm", "n": 32, "dim": 4096, "group": 128, "residual": True, "y": False},
        # a prompt chunk's residual stream, with the BF16 value too
        {"name": "norm: prefill chunk", "op": "norm", "n": 8191, "dim": 7168, "group": 128, "residual": True, "y": True},
        # the indexer heads' queries of a prompt chunk, two scales of 64 values each
        {"name": "norm: indexer heads", "op": "norm", "n": 262144, "dim": 128, "group": 64, "residual": False, "y": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attn", "attn", "beam", "compact", "norm"])
    if op == "cache":
        seqs = rng.randint(1, 32)
        n = min(_log(rng, 1, 65000), seqs * 2048)
        return {"op": op, "n": n, "seqs": seqs, "entries": max(2048, -(-n // seqs)), "spread": round(rng.uniform(0, 6), 2)}
    if op == "attn":
        H = rng.choice([rng.randint(1, 128), 16, 64, 128])
        kc = _log(rng, 1, 2048)
        kw = rng.choice([0, 16, 128, rng.randint(1, 256)])
        most = max(1, 4096 * 640 * 64 // ((kc + kw) * H))
        T = _log(rng, 1, min(4096, most))
        mode = "prefill" if T > 256 else rng.choice(["decode", "decode", "prefill"])
        N = max(kc, _log(rng, 256, 16384))
        return {"op": op, "mode": mode, "T": T, "H": H, "N": N, "kc": kc, "kw": kw,
                "fill": rng.choice(["full", "ragged"]), "sharp": round(rng.uniform(0.5, 4.0), 2)}
    if op == "beam":
        return {"op": op, "seqs": _log(rng, 1, 64), "width": rng.randint(1, 6), "tokens": _log(rng, 1, 16384),
                "kinds": rng.choice(["kv_fp4,idxk_fp4", "kv,idxk", "kv_fp4,idxk", "kv_fp4"]),
                "slack": round(rng.uniform(1.05, 2.0), 2)}
    if op == "compact":
        return {"op": op, "pages": _log(rng, 3, 40000), "used": round(rng.uniform(0.05, 0.98), 3), "rows": _log(rng, 1, 128),
                "kinds": rng.choice(["kv_fp4,idxk_fp4", "kv_fp4", "kv_fp4,idxk", "idxk_fp4"])}
    group = rng.choice([64, 128])
    dim = group * _log(rng, 1, 8192 // group)
    return {"op": op, "n": max(1, min(_log(rng, 1, 65536), 50_000_000 // dim)), "dim": dim, "group": group,
            "residual": rng.random() < 0.6, "y": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _pool(kind, pages):
    """A zeroed pool of `pages` pages whose first byte is 1024-byte aligned."""
    nbytes = pages * page_bytes(kind)
    buf = torch.zeros(nbytes + 1024, dtype=torch.uint8, device=DEV)
    off = -buf.data_ptr() % 1024
    return buf[off:off + nbytes].view(pages, page_bytes(kind))


def _blocks(pool, kind):
    """The page's blocks as views [pages, 64, bytes per slot]."""
    out, at = [], 0
    for rb in BLOCKS[kind]:
        out.append(pool[:, at:at + PAGE * rb].unflatten(1, (PAGE, rb)))
        at += PAGE * rb
    return out


def _fp4_pages(g, pages):
    """A KV_FP4 pool of rows drawn from N(0, 1) (block exponents -2 .. -1, as such rows get)."""
    pool = _pool("kv_fp4", pages)
    codes, rope, scale = _blocks(pool, "kv_fp4")
    for a in range(0, pages, 512):
        b = min(pages, a + 512)
        x = _randn(g, b - a, PAGE, DIM).to(torch.bfloat16)
        c, e, r = _quantise(x.view(-1, DIM))
        codes[a:b] = c.view(b - a, PAGE, 224)
        scale[a:b, :, :14] = e.view(b - a, PAGE, 14)
        rope[a:b] = r.view(b - a, PAGE, 128)
    return pool


def _page_table(g, seqs, per_seq, pages):
    return torch.randperm(pages, generator=g, device=DEV)[:seqs * per_seq].view(seqs, per_seq).to(torch.int32)


def _distinct(g, T, N, k):
    """k distinct entries below N for each of T rows, ascending, int32 [T, k]."""
    out = torch.empty(T, k, dtype=torch.int32, device=DEV)
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        out[a:b] = torch.rand(b - a, N, generator=g, device=DEV).topk(k, dim=1).indices.sort(dim=1).values
    return out


def _lib():
    from compressed_sparse_attention_c4_gb300 import dsv4sa
    return dsv4sa


def prepare(case, seed):
    g = _gen(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    s["op"] = case["op"]
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps beside its buffers: the pools' descriptors."""
    L = _lib()
    desc = lambda kind, pool: L.dsv4sa_pool_desc_init(KINDS[kind], pool, pool.shape[0])  # noqa: E731
    if s["op"] == "cache":
        s["desc"] = desc("kv_fp4", s["pool"])
    elif s["op"] == "attn":
        s["comp_desc"], s["win_desc"] = desc("kv_fp4", s["comp"]), desc("kv_fp4", s["win"])
    elif s["op"] in ("beam", "compact"):
        s["cache"] = L.page_cache([desc(k, p) for k, p in zip(s["kinds"], s["pools"])], s["table"], s["use"])
        if s["op"] == "compact":
            s["dst_cache"] = L.page_cache([desc(k, p) for k, p in zip(s["kinds"], s["dst_pools"])], s["dst_table"],
                                          s["dst_use"])


def _prepare_cache(case, g):
    n, seqs = case["n"], case["seqs"]
    per = -(-case["entries"] // PAGE)
    pages = seqs * per + 3
    table = _page_table(g, seqs, per, pages)
    # each sequence's next rows, the sequences in turn, from an arbitrary entry on
    i = torch.arange(n, device=DEV)
    start = torch.randint(0, max(1, per * PAGE - -(-n // seqs) + 1), (seqs,), generator=g, device=DEV)
    seq = i % seqs
    rows = _randn(g, n, DIM) * torch.exp2(case["spread"] * _randn(g, n, DIM // 32).repeat_interleave(32, 1))
    return {"pool": _pool("kv_fp4", pages), "table": table, "row_seq": seq.to(torch.int32),
            "row_entry": (start[seq] + i // seqs).to(torch.int32), "rows": rows.to(torch.bfloat16),
            "back": torch.empty(n, DIM, dtype=torch.bfloat16, device=DEV)}


def _prepare_attn(case, g):
    T, H, N, kc, kw = case["T"], case["H"], case["N"], case["kc"], case["kw"]
    decode = case["mode"] == "decode"
    seqs = T if decode else 1
    per = -(-N // PAGE)
    comp_pages = seqs * per + 2
    idx = _distinct(g, T, N, kc)
    if decode:   # a ring of window slots for each sequence
        ring = -(-max(kw, 1) // PAGE) * PAGE
        pos = torch.randint(ring, 4 * N + ring, (T,), generator=g, device=DEV).to(torch.int32)
        win_per = ring // PAGE
    else:        # the prompt chunk's last tokens, all of one sequence
        ring = 0
        pos = torch.arange(4 * N - T, 4 * N, device=DEV).clamp(min=0).to(torch.int32)
        win_per = -(-4 * N // PAGE)
    if case["fill"] == "ragged":   # rows shorter than kc, and one in twenty with nothing at all
        keep = (torch.rand(T, generator=g, device=DEV) ** 2 * (kc + 1)).to(torch.int32)
        empty = torch.rand(T, generator=g, device=DEV) < 0.05
        keep = torch.where(empty, torch.zeros_like(keep), keep)
        idx = torch.where(torch.arange(kc, device=DEV)[None] < keep[:, None], idx, -1)
        pos = torch.where(empty, -1, pos)                       # no window position is visible
        pos = torch.where((torch.rand(T, generator=g, device=DEV) < 0.2) & ~empty, pos % max(kw, 1), pos)
    win_pages = seqs * win_per + 2
    return {"mode": case["mode"], "q": (case["sharp"] * _randn(g, T, H, DIM)).to(torch.bfloat16), "sink": _randn(g, H),
            "q_seq": (torch.arange(T, device=DEV) if decode else torch.zeros(T, device=DEV)).to(torch.int32),
            "comp": _fp4_pages(g, comp_pages), "comp_pt": _page_table(g, seqs, per, comp_pages),
            "win": _fp4_pages(g, win_pages), "win_pt": _page_table(g, seqs, win_per, win_pages),
            "idx": idx.contiguous(), "pos": pos.to(torch.int32), "kw": kw, "ring": ring,
            "out": torch.empty(T, H, DIM, dtype=torch.bfloat16, device=DEV),
            "lse": torch.empty(T, H, dtype=torch.float32, device=DEV)}


def _prepare_beam(case, g):
    seqs, width = case["seqs"], case["width"]
    kinds = case["kinds"].split(",")
    # one compressed entry for four tokens; lengths differ a little, some end with a page
    length = -(-case["tokens"] // 4) - torch.randint(0, 64, (seqs,), generator=g, device=DEV)
    length = length.clamp(min=0)
    per = int(-(-case["tokens"] // 4) // PAGE) + 1
    used = seqs * per + 2 * seqs * width
    pages = int(used * case["slack"]) + 2
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    rows = seqs * (1 + width)
    table = torch.full((rows, per + 1), -1, dtype=torch.int32, device=DEV)
    n_pg = (length + PAGE - 1) // PAGE
    col = torch.arange(per + 1, device=DEV)
    own_pg = perm[:seqs * (per + 1)].view(seqs, per + 1) if pages >= seqs * (per + 1) else perm[:seqs * per].view(seqs, per)
    own_pg = torch.nn.functional.pad(own_pg, (0, per + 1 - own_pg.shape[1]), value=-1)
    table[:seqs] = torch.where(col[None] < n_pg[:, None], own_pg, -1)
    # the last step's forks, of other parents: their full pages are shared
    parent = torch.randint(0, seqs, (seqs * width,), generator=g, device=DEV)
    table[seqs:] = torch.where(col[None] < (length[parent] // PAGE)[:, None], table[parent], -1)
    use = torch.zeros(pages, dtype=torch.int32, device=DEV)
    flat = table.reshape(-1)
    use.scatter_add_(0, flat.clamp(min=0).long(), (flat >= 0).to(torch.int32))
    src = torch.arange(seqs, device=DEV).repeat_interleave(width)[torch.randperm(seqs * width, generator=g, device=DEV)]
    pools = []
    for k in kinds:
        p = _pool(k, pages)
        p.copy_(torch.randint(0, 256, p.shape, generator=g, device=DEV, dtype=torch.uint8))
        pools.append(p)
    dst = torch.arange(seqs, rows, device=DEV).to(torch.int32)
    return {"kinds": kinds, "pools": pools, "table": table, "use": use, "src": src.to(torch.int32), "dst": dst,
            "len": length[src].to(torch.int32), "new": torch.empty(seqs * width, dtype=torch.int32, device=DEV)}


def _prepare_compact(case, g):
    P, rows = case["pages"], case["rows"]
    kinds = case["kinds"].split(",")
    n_used = max(1, int(P * case["used"]))
    ids = torch.randperm(P, generator=g, device=DEV)[:n_used].to(torch.int32)
    per = -(-n_used // rows) + 5
    table = torch.full((rows, per), -1, dtype=torch.int32, device=DEV)
    fill = torch.full((rows, per - 5), -1, dtype=torch.int32, device=DEV)
    fill.view(-1)[:n_used] = ids
    table[:, :per - 5] = fill
    shared = torch.randint(0, n_used, (rows, 4), generator=g, device=DEV)     # some pages of every row are shared
    table[:, per - 5:per - 1] = ids[shared]
    use = torch.zeros(P, dtype=torch.int32, device=DEV)
    flat = table.reshape(-1)
    use.scatter_add_(0, flat.clamp(min=0).long(), (flat >= 0).to(torch.int32))
    pools, dst = [], []
    for k in kinds:
        p = _pool(k, P)
        p.copy_(torch.randint(0, 256, p.shape, generator=g, device=DEV, dtype=torch.uint8))
        pools.append(p)
        dst.append(_pool(k, n_used + 1))
    return {"kinds": kinds, "pools": pools, "table": table, "use": use, "dst_pools": dst,
            "dst_table": torch.empty_like(table), "dst_use": torch.empty(n_used + 1, dtype=torch.int32, device=DEV),
            "new_id": torch.empty(P, dtype=torch.int32, device=DEV),
            "n_used": torch.empty(1, dtype=torch.int32, device=DEV)}


def _prepare_norm(case, g):
    n, dim, group = case["n"], case["dim"], case["group"]
    x = torch.empty(n, dim, dtype=torch.bfloat16, device=DEV)
    r = torch.empty_like(x) if case["residual"] else None
    heavy = torch.exp2(1.5 * _randn(g, dim))          # a few features of a residual stream are much larger
    for a in range(0, n, 65536):
        b = min(n, a + 65536)
        x[a:b] = (_randn(g, b - a, dim) * heavy).to(torch.bfloat16)
        if r is not None:
            r[a:b] = (4 * _randn(g, b - a, dim) * heavy).to(torch.bfloat16)
    return {"x": x, "residual": r, "w": 1 + 0.2 * _randn(g, dim), "eps": 1e-6, "group": group,
            "sum": torch.empty_like(x) if r is not None else None, "y": torch.empty_like(x) if case["y"] else None,
            "codes": torch.empty(n, dim, dtype=torch.uint8, device=DEV),
            "scale": torch.empty(n, dim // group, dtype=torch.float32, device=DEV)}


# ------------------------------------------------------------------ one pass

def run(s):
    return globals()[("_own_" if own else "_plain_") + s["op"]](s)


def _own_cache(s):
    L = _lib()
    L.dsv4sa_cache_write(s["desc"], s["table"], s["row_seq"], s["row_entry"], s["rows"])
    L.dsv4sa_cache_read(s["desc"], s["table"], s["row_seq"], s["row_entry"], s["back"])
    return {"rows": s["back"], "pool": s["pool"].view(torch.int32)}


def _own_attn(s):
    L = _lib()
    fn = L.dsv4sa_sparse_attn_decode if s["mode"] == "decode" else L.dsv4sa_sparse_attn_prefill
    fn(s["q"], s["sink"], s["q_seq"], s["comp_desc"], s["comp_pt"], s["idx"], s["win_desc"], s["win_pt"], None, s["out"],
       SOFTMAX_SCALE, lse=s["lse"], win_pos=s["pos"], kw=s["kw"], win_ring=s["ring"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_beam(s):
    L = _lib()
    L.dsv4sa_cache_release(s["cache"], s["dst"])
    L.dsv4sa_cache_fork(s["cache"], s["src"], s["dst"], s["len"], s["new"])
    return {"table": s["table"], "use": s["use"], "new": s["new"], "pools": [p.view(torch.int32) for p in s["pools"]]}


def _own_compact(s):
    L = _lib()
    L.dsv4sa_cache_compact(s["cache"], s["dst_cache"], s["new_id"], s["n_used"])
    return {"table": s["dst_table"], "use": s["dst_use"], "new_id": s["new_id"], "n_used": s["n_used"],
            "pools": [p.view(torch.int32) for p in s["dst_pools"]]}


def _own_norm(s):
    L = _lib()
    L.dsv4sa_rmsnorm_quant(s["x"], s["w"], s["codes"], s["scale"], group=s["group"], residual=s["residual"],
                           residual_out=s["sum"], y=s["y"], eps=s["eps"])
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"],
            **({"sum": s["sum"]} if s["sum"] is not None else {}), **({"y": s["y"]} if s["y"] is not None else {})}


# ------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], by its bits."""
    e = e.to(torch.int32)
    return torch.where(e == -127, 0x00400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """BF16 rows [n, 512] -> (packed E2M1 codes [n, 224], E8M0 bytes [n, 14], rope bytes [n, 128])."""
    n = x.shape[0]
    v = x[:, :NOPE].float().view(n, 14, 32)
    amax = v.abs().amax(-1).clamp(min=6.0 * 2.0 ** -126)
    m, e = torch.frexp(amax * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device))   # m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)                                                        # ceil(log2)
    y = (v * _pow2(-e)[..., None]).clamp(-6, 6)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).view(n, NOPE)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return packed, (e + 127).to(torch.uint8), x[:, NOPE:].contiguous().view(torch.uint8)


def _dequantise(codes, scale, rope):
    """Bytes of rows -> fp32 values [..., 512]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    f = _pow2(scale[..., :14].to(torch.int32) - 127)
    nope = lut[c] * f.repeat_interleave(32, dim=-1)
    return torch.cat((nope, rope.contiguous().view(torch.bfloat16).float()), dim=-1)


def _slots(table, seq, entry):
    e = entry.long().clamp(min=0)
    return table[seq.long(), e // PAGE].long(), e % PAGE


def _plain_cache(s):
    codes, rope, scale = _blocks(s["pool"], "kv_fp4")
    page, slot = _slots(s["table"], s["row_seq"], s["row_entry"])
    c, e, r = _quantise(s["rows"])
    codes[page, slot] = c
    rope[page, slot] = r
    scale[..., :14][page, slot] = e
    back = _dequantise(codes[page, slot], scale[page, slot], rope[page, slot]).to(torch.bfloat16)
    return {"rows": back, "pool": s["pool"].view(torch.int32)}


def _window(s, a, b):
    p = s["pos"][a:b].long()[:, None] - s["kw"] + 1 + torch.arange(s["kw"], device=DEV)
    ok = p >= 0
    return (p % s["ring"] if s["ring"] else p).clamp(min=0), ok


def _rows(pool, table, seq, entry):
    codes, rope, scale = _blocks(pool, "kv_fp4")
    page, slot = _slots(table, seq[:, None], entry)
    return _dequantise(codes[page, slot], scale[page, slot], rope[page, slot])


def _plain_attn(s):
    T, H = s["q"].shape[:2]
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    R = s["idx"].shape[1] + s["kw"]
    step = max(1, min(T, 2 ** 27 // (R * DIM)))
    for a in range(0, T, step):
        b = min(T, a + step)
        seq, idx = s["q_seq"][a:b], s["idx"][a:b]
        kv, ok = _rows(s["comp"], s["comp_pt"], seq, idx), idx >= 0
        if s["kw"]:
            p, pok = _window(s, a, b)
            kv, ok = torch.cat((kv, _rows(s["win"], s["win_pt"], seq, p)), 1), torch.cat((ok, pok), 1)
        x = torch.bmm(s["q"][a:b].float(), kv.transpose(1, 2)) * SOFTMAX_SCALE
        x = x.masked_fill(~ok[:, None, :], -math.inf)
        m = torch.maximum(x.amax(-1), s["sink"][None])
        p = torch.exp(x - m[..., None])
        z = p.sum(-1) + torch.exp(s["sink"][None] - m)
        kv = kv * ok[..., None]
        out[a:b] = (torch.bmm(p, kv) / z[..., None]).to(torch.bfloat16)
        lse[a:b] = m + torch.log(z)
    return {"out": out, "lse": lse}


def _plain_beam(s):
    table, use = s["table"], s["use"]
    old = table[s["dst"].long()]
    use.scatter_add_(0, old.clamp(min=0).long().view(-1), -(old >= 0).to(torch.int32).view(-1))
    n, cols = s["src"].shape[0], table.shape[1]
    full, part = s["len"].long() // PAGE, s["len"].long() % PAGE
    free = torch.nonzero(use == 0).view(-1)
    rank = torch.cumsum(part > 0, 0) - 1
    new = torch.where(part > 0, free[rank.clamp(min=0)], -1)
    col = torch.arange(cols, device=DEV)
    src = table[s["src"].long()]
    shared = torch.where(col < full[:, None], src, -1)
    table[s["dst"].long()] = torch.where((col == full[:, None]) & (part > 0)[:, None], new[:, None].to(torch.int32), shared)
    use.scatter_add_(0, shared.clamp(min=0).long().view(-1), (shared >= 0).to(torch.int32).view(-1))
    at = torch.nonzero(part > 0).view(-1)
    use[new[at]] = 1
    if at.numel():
        last = src[at, full[at]].long()
        keep = (torch.arange(PAGE, device=DEV) < part[at][:, None])[..., None]
        for kind, pool in zip(s["kinds"], s["pools"]):
            for blk in _blocks(pool, kind):
                blk[new[at]] = torch.where(keep, blk[last], blk[new[at]])
    s["new"].copy_(new)
    return {"table": table, "use": use, "new": s["new"], "pools": [p.view(torch.int32) for p in s["pools"]]}


def _plain_compact(s):
    used = s["use"] > 0
    new_id = torch.where(used, torch.cumsum(used, 0) - 1, -1).to(torch.int32)
    ids = torch.nonzero(used).view(-1)
    for p, d in zip(s["pools"], s["dst_pools"]):
        d[:ids.shape[0]] = p[ids]
    t = s["table"]
    s["dst_table"].copy_(torch.where(t >= 0, new_id[t.clamp(min=0).long()], -1))
    s["dst_use"].zero_()
    s["dst_use"][:ids.shape[0]] = s["use"][ids]
    return {"table": s["dst_table"], "use": s["dst_use"], "new_id": new_id,
            "n_used": used.sum(dtype=torch.int32).view(1), "pools": [d.view(torch.int32) for d in s["dst_pools"]]}


def _plain_norm(s):
    n, dim = s["x"].shape
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    h = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["w"]
    blk = h.view(n, dim // s["group"], s["group"])
    scale = blk.abs().amax(-1).clamp(min=1e-4) * torch.tensor(1.0 / 448.0, dtype=torch.float32, device=DEV)
    codes = (blk / scale[..., None]).clamp(-448, 448).view(n, dim).to(torch.float8_e4m3fn)
    return {"codes": codes, "scale": scale, **({"sum": v.to(torch.bfloat16)} if s["sum"] is not None else {}),
            **({"y": h.to(torch.bfloat16)} if s["y"] is not None else {})}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] in ("beam", "compact"):
        return None          # copies and counts: whole numbers
    s = globals()["_prepare_" + case["op"]](case, _gen(seed))
    return globals()["_exact_" + case["op"]](s)


def _grid():
    return torch.tensor(sorted(set(E2M1) | {-v for v in E2M1}), dtype=torch.float64, device=DEV)


def _exact_cache(s):
    """Each block of 32 values on the E2M1 grid times the smallest power of two that covers it."""
    out = s["rows"].double()
    grid = _grid()
    even = torch.tensor([abs(float(v)) in (0.0, 1.0, 2.0, 4.0) for v in grid], device=DEV)   # mantissa bit clear
    for a in range(0, out.shape[0], 4096):
        v = out[a:a + 4096, :NOPE].reshape(-1, 32)
        top = v.abs().amax(-1).clamp(min=6.0 * 2.0 ** -126)
        m, e = torch.frexp(top / 6.0)
        e = torch.where(m == 0.5, e - 1, e).long()                  # the smallest e with 6 * 2^e >= top
        step = ((e + 1023) << 52).view(torch.float64)
        y = (v / step[:, None]).clamp(-6, 6)
        hi = torch.searchsorted(grid, y).clamp(1, grid.numel() - 1)
        lo = hi - 1
        dl, dh = y - grid[lo], grid[hi] - y
        pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(even[lo], lo, hi)))
        out[a:a + 4096, :NOPE] = (grid[pick] * step[:, None]).view(-1, NOPE)
    return {"rows": out, "pool": None}


def _exact_attn(s):
    T, H = s["q"].shape[:2]
    kc, kw = s["idx"].shape[1], s["kw"]
    value = {}
    for name in ("comp", "win"):     # every row of the pools, dequantised once
        codes, rope, scale = _blocks(s[name], "kv_fp4")
        P = s[name].shape[0]
        nib = torch.empty(P, PAGE, NOPE, dtype=torch.int64, device=DEV)
        nib[..., 0::2], nib[..., 1::2] = (codes % 16).long(), (codes // 16).long()
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[nib % 8]
        val = torch.where(nib >= 8, -mag, mag).view(P, PAGE, 14, 32) * ((scale[..., :14].long() - 127 + 1023) << 52).view(torch.float64)[..., None]
        full = torch.empty(P * PAGE, DIM, dtype=torch.float32, device=DEV)      # exact: 2 significant bits
        full[:, :NOPE] = val.view(-1, NOPE)
        full[:, NOPE:] = rope.contiguous().view(torch.bfloat16).view(-1, ROPE)
        value[name] = full
        del nib, mag, val
    out = torch.empty(T, H, DIM, dtype=torch.float64, device=DEV)
    lse = torch.empty(T, H, dtype=torch.float64, device=DEV)
    step = max(1, 2 ** 25 // ((kc + kw) * DIM))
    for a in range(0, T, step):
        b = min(T, a + step)
        seq = s["q_seq"][a:b].long()
        parts = []
        e = s["idx"][a:b].long()
        parts.append(("comp", torch.gather(s["comp_pt"][seq].long(), 1, e.clamp(min=0) // PAGE) * PAGE + e.clamp(min=0) % PAGE,
                      e >= 0))
        if kw:
            p = s["pos"][a:b].long()[:, None] - (kw - 1) + torch.arange(kw, device=DEV)
            e = torch.where(p < 0, 0, p % s["ring"] if s["ring"] else p)
            parts.append(("win", torch.gather(s["win_pt"][seq].long(), 1, e // PAGE) * PAGE + e % PAGE, p >= 0))
        kv = torch.cat([value[n][i].double() * ok[..., None] for n, i, ok in parts], 1)
        ok = torch.cat([ok for _, _, ok in parts], 1)
        x = torch.einsum("thd,trd->thr", s["q"][a:b].double(), kv) * SOFTMAX_SCALE
        x = torch.cat((torch.where(ok[:, None], x, -math.inf), s["sink"].double().expand(b - a, H)[..., None]), -1)
        z = torch.logsumexp(x, -1)
        out[a:b] = torch.einsum("thr,trd->thd", torch.exp(x[..., :-1] - z[..., None]), kv)
        lse[a:b] = z
    return {"out": out, "lse": lse}


def _e4m3(v):
    """fp64 -> the nearest E4M3 value, ties to even, as fp64."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    q = torch.exp2(e - 3)
    return (torch.round(v / q) * q).clamp(-448, 448)


def _exact_norm(s):
    n, dim = s["x"].shape
    total = torch.empty(n, dim, dtype=torch.float64, device=DEV)
    codes = torch.empty_like(total)
    y = torch.empty_like(total) if s["y"] is not None else None
    scale = torch.empty(s["scale"].shape, dtype=torch.float64, device=DEV)
    w = s["w"].double()
    for a in range(0, n, 8192):
        b = min(n, a + 8192)
        v = s["x"][a:b].double()
        if s["residual"] is not None:
            v = v + s["residual"][a:b].double()
        total[a:b] = v
        h = v / torch.sqrt(torch.sum(v * v, -1, keepdim=True) / dim + s["eps"]) * w
        if y is not None:
            y[a:b] = h
        h = h.view(b - a, -1, s["group"])
        top = h.abs().amax(-1).clamp(min=1e-4) / 448.0
        scale[a:b] = top
        codes[a:b] = _e4m3(h / top[..., None]).view(b - a, dim)
    return {"codes": codes, "scale": scale, **({"sum": total} if s["sum"] is not None else {}),
            **({"y": y} if y is not None else {})}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "cache":
        # each BF16 row read and its packed row written, the packed row read and its BF16 values written
        return {"bytes": case["n"] * (1024 + 366 + 8 + 366 + 1024), "flops": 6 * case["n"] * DIM}
    if op == "attn":
        T, H, kc, kw = case["T"], case["H"], case["kc"], case["kw"]
        share = 0.33 if case["fill"] == "ragged" else 1.0
        seqs = T if case["mode"] == "decode" else 1
        rows = min(T * kc * share, seqs * case["N"]) + (T * kw if case["mode"] == "decode" else min(T + kw, 4 * case["N"]))
        return {"bytes": int(T * H * (1024 + 1024 + 4) + rows * 366 + T * kc * 4),
                "flops": int(4 * T * H * DIM * (kc * share + kw * (0.85 if case["fill"] == "ragged" else 1.0)))}
    kinds = [BLOCKS[k] for k in case["kinds"].split(",")] if "kinds" in case else []
    slot = sum(sum(k) for k in kinds)
    if op == "beam":
        forks, per = case["seqs"] * case["width"], case["tokens"] // 4 // PAGE + 2
        # half a page copied on average, every fork's table row released and written, a use count for each page
        return {"bytes": forks * (2 * slot * PAGE // 2 + per * 4 * 3) + case["seqs"] * per * 4 * 2, "flops": 0}
    if op == "compact":
        used = max(1, int(case["pages"] * case["used"]))
        return {"bytes": 2 * used * slot * PAGE + case["pages"] * 8 + used * 12, "flops": 0}
    n, dim = case["n"], case["dim"]
    per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
    return {"bytes": n * dim * per + n * (dim // case["group"]) * 4 + dim * 4, "flops": 8 * n * dim}
