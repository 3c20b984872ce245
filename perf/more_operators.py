"""The library's operators around a step of speculative decoding, as cases to measure.

Three groups of calls, each as a serving program makes them:

* ``table``, ``rope``  the (cos, sin) table of a long context, and queries normed per head and rotated
  (the last 64 dims of the attention's heads, pairs side by side; half of an indexer head, its two
  halves paired);
* ``append``  new rows of the KV projection normed, rotated at their positions, quantised and put into
  their slots: the ring of raw tokens or consecutive entries, FP8 or FP4;
* ``tree``  attention of drafted tokens, a tree or a chain of them a sequence, over every compressed
  entry, the committed window and the drafted ancestors; ``list`` the window list of each drafted token,
  for the attention of layers whose indexer selects entries.

``run`` computes the plain form in elementary torch operations, or, with ``own`` set, makes the
library's calls.  ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 64
NOPE, ROPE, DIM = 448, 64, 512
WINDOW, RING, DRAFT = 128, 128, 128      # raw tokens a query sees; ring slots; first slot of drafted rows
KINDS = {"kv": 0, "kv_fp4": 3}
# bytes per slot of each block of a page, in the order the blocks lie in it
BLOCKS = {"kv": (448, 128, 32), "kv_fp4": (224, 128, 16)}
ROW_BYTES = {"kv": 604, "kv_fp4": 366}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SOFTMAX_SCALE = 1.0 / math.sqrt(512.0)
EPS = 1e-6
# rotary base of the raw tokens and of the compressed layers, and a context scaled 16 times
YARN = {"base": 160000.0, "factor": 16.0, "original_len": 65536, "beta_fast": 32.0, "beta_slow": 1.0}


def page_bytes(kind):
    return PAGE * sum(BLOCKS[kind])


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the table of a context of a million tokens, made once when a program starts
        {"name": "table: 1M positions", "op": "table", "rows": 1048576, "pairs": 32, "first": 0},
        # a decode batch's queries, 64 heads each: normed and rotated
        {"name": "rope: decode queries", "op": "rope", "T": 32, "H": 64, "dim": 512, "rope": 64, "halves": False, "norm": True},
        # a prompt chunk's queries
        {"name": "rope: prompt queries", "op": "rope", "T": 4096, "H": 64, "dim": 512, "rope": 64, "halves": False,
         "norm": True},
        # the indexer heads of a prompt chunk, the pairs in two halves
        {"name": "rope: indexer heads", "op": "rope", "T": 8191, "H": 64, "dim": 128, "rope": 64, "halves": True, "norm": False},
        # one decode step of 32 sequences: a row each into the ring of raw tokens
        {"name": "append: decode batch", "op": "append", "n": 32, "seqs": 32, "kind": "kv", "norm": True, "ring": True},
        # a long prompt's rows at once
        {"name": "append: long prompt", "op": "append", "n": 65529, "seqs": 4, "kind": "kv", "norm": True, "ring": False},
        # rows normed before, into a 4-bit cache
        {"name": "append: 4-bit cache", "op": "append", "n": 32749, "seqs": 3, "kind": "kv_fp4", "norm": False, "ring": False},
        # one token over a short context, where latency is all
        {"name": "tree: one token", "op": "tree", "seqs": 1, "nodes": 1, "shape": "chain", "H": 16, "N": 512,
         "fill": "full", "kind": "kv"},
        # four tokens in a row for each of 32 sequences of 64K tokens
        {"name": "tree: chains at 64K", "op": "tree", "seqs": 32, "nodes": 4, "shape": "chain", "H": 64,
         "N": 512, "fill": "full", "kind": "kv"},
        # a mixed batch of trees over short and long contexts, 4-bit cache, a sequence without tokens, rows behind the last
        {"name": "tree: mixed batch", "op": "tree", "seqs": 64, "nodes": 13, "shape": "tree", "H": 8,
         "N": 8192, "fill": "ragged", "kind": "kv_fp4"},
        # trees of 16 at the end of a million tokens
        {"name": "tree: trees at 1M", "op": "tree", "seqs": 8, "nodes": 16, "shape": "tree", "H": 64,
         "N": 8192, "fill": "full", "kind": "kv"},
        # the window lists of trees of 24 for a batch of 128
        {"name": "list: trees of a batch", "op": "list", "seqs": 128, "nodes": 24, "shape": "tree", "fill": "ragged"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "append", "append", "tree", "tree", "tree", "list"])
    if op == "table":
        return {"op": op, "rows": _log(rng, 1, 1000000), "pairs": rng.choice([16, 32, 32, 64]), "first": rng.choice([0, _log(rng, 1, 1000000)])}
    if op == "rope":
        H = rng.choice([rng.randint(1, 128), 1, 64])
        dim = rng.choice([512, 128, 8 * rng.randint(4, 64)])
        rope = 16 * rng.randint(1, min(dim // 16, 8))
        T = _log(rng, 1, max(1, min(16384, 4096 * 64 * 512 // (H * dim))))
        return {"op": op, "T": T, "H": H, "dim": dim, "rope": rope, "halves": rng.random() < 0.5, "norm": rng.random() < 0.5}
    if op == "append":
        kind = rng.choice(["kv", "kv", "kv_fp4"])
        seqs = rng.randint(1, 64)
        ring = rng.random() < 0.4
        n = min(_log(rng, 1, 65000), seqs * (RING if ring else 16384))
        return {"op": op, "n": n, "seqs": seqs, "kind": kind, "norm": kind == "kv" and rng.random() < 0.6, "ring": ring}
    nodes = rng.choice([1, rng.randint(1, 64), rng.randint(2, 16)])
    shape, fill = rng.choice(["chain", "tree"]), rng.choice(["full", "ragged"])
    if op == "list":
        return {"op": op, "seqs": _log(rng, 1, 256), "nodes": nodes, "shape": shape, "fill": fill}
    H = rng.choice([rng.randint(1, 128), 8, 16, 64])
    N = _log(rng, 1, 8192)
    most = max(1, min(64, 8 * 16 * 64 * 8320 // (nodes * H * (N + WINDOW))))
    return {"op": op, "seqs": _log(rng, 1, most), "nodes": nodes, "shape": shape, "H": H, "N": N, "fill": fill,
            "kind": rng.choice(["kv", "kv_fp4"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


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


def _random_pages(g, kind, pages):
    """A pool of rows drawn from N(0, 1), quantised."""
    pool = _pool(kind, pages)
    codes, rope, scale = _blocks(pool, kind)
    for a in range(0, pages, 512):
        b = min(pages, a + 512)
        x = _randn(g, (b - a) * PAGE, DIM).to(torch.bfloat16)
        c, s = _quantise(x[:, :NOPE].float(), kind)
        codes[a:b] = c.view(b - a, PAGE, -1)
        scale[a:b, :, :s.shape[-1]] = s.view(b - a, PAGE, -1)
        rope[a:b] = x[:, NOPE:].contiguous().view(torch.uint8).view(b - a, PAGE, 128)
    return pool


def _page_table(g, seqs, per_seq, pages):
    return torch.randperm(pages, generator=g, device=DEV)[:seqs * per_seq].view(seqs, per_seq).to(torch.int32)


def _frequencies(pairs, base, factor, original_len, beta_fast, beta_slow):
    """Angle a position of each pair (fp64), the low ones divided by `factor` as YaRN does."""
    d = 2 * pairs
    w = base ** (-np.arange(pairs, dtype=np.float64) * 2 / d)
    if factor == 1.0:
        return w
    at = [d * math.log(original_len / (beta * 2 * math.pi)) / (2 * math.log(base)) for beta in (beta_fast, beta_slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
    keep = 1 - np.clip((np.arange(pairs) - lo) / max(hi - lo, 1e-3), 0, 1)
    return w / factor * (1 - keep) + w * keep


def _table(first, rows, pairs):
    w = torch.from_numpy(_frequencies(pairs, **YARN)).to(DEV)
    out = torch.empty(rows, pairs, 2, dtype=torch.float32, device=DEV)
    for a in range(0, rows, 131072):
        b = min(rows, a + 131072)
        ang = torch.arange(first + a, first + b, device=DEV, dtype=torch.float64)[:, None] * w
        out[a:b, :, 0], out[a:b, :, 1] = torch.cos(ang), torch.sin(ang)
    return out


def _lib():
    from compressed_sparse_attention_c4_gb300 import dsv4sa
    return dsv4sa


def prepare(case, seed):
    g = _gen(seed)
    s = globals()["_prepare_" + case["op"]](case, g, seed)
    s["op"] = case["op"]
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps beside its buffers: pool descriptors, workspaces."""
    L = _lib()
    desc = lambda pool: L.dsv4sa_pool_desc_init(KINDS[s["kind"]], pool, pool.shape[0])  # noqa: E731
    if s["op"] == "append":
        s["desc"] = desc(s["pool"])
    elif s["op"] == "tree":
        s["comp_desc"], s["win_desc"] = desc(s["comp"]), desc(s["win"])
        nbytes = L.dsv4sa_tree_attn_workspace_size(len(s["seqs"]), s["max_nodes"], s["q"].shape[1], s["n_max"], WINDOW)
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None


def _prepare_table(case, g, seed):
    first = case["first"] + seed % 1000
    return {"first": first, "cs": torch.empty(case["rows"], case["pairs"], 2, dtype=torch.float32, device=DEV)}


def _prepare_rope(case, g, seed):
    T, H, dim = case["T"], case["H"], case["dim"]
    x = torch.empty(T, H, dim, dtype=torch.bfloat16, device=DEV)
    heavy = torch.exp2(_randn(g, dim))                   # some features of a projection are larger
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        x[a:b] = (_randn(g, b - a, H, dim) * heavy).to(torch.bfloat16)
    rows = 65536
    pos = torch.randint(0, rows, (T,), generator=g, device=DEV) if T <= 256 else (
        torch.arange(T, device=DEV) + int(torch.randint(0, rows - T + 1, (1,), generator=g, device=DEV)))
    return {"x": x, "cs": _table(0, rows, case["rope"] // 2), "pos": pos.to(torch.int32), "rope": case["rope"], "halves": case["halves"],
            "norm": case["norm"], "out": torch.empty_like(x)}


def _prepare_append(case, g, seed):
    n, seqs, kind = case["n"], case["seqs"], case["kind"]
    per = RING // PAGE if case["ring"] else -(-max(n, 2048) // seqs // PAGE) + 2
    pages = seqs * per + 3
    # each sequence's next rows, the sequences in turn, from an arbitrary position on
    i = torch.arange(n, device=DEV)
    most = per * PAGE - -(-n // seqs) if not case["ring"] else 60000
    start = torch.randint(0, max(1, most + 1), (seqs,), generator=g, device=DEV)
    seq = i % seqs
    pos = start[seq] + i // seqs
    heavy = torch.exp2(_randn(g, DIM))
    rows = (_randn(g, n, DIM) * heavy).to(torch.bfloat16)
    return {"kind": kind, "pool": _pool(kind, pages), "table": _page_table(g, seqs, per, pages), "row_seq": seq.to(torch.int32),
            "row_pos": pos.to(torch.int32), "rows": rows, "cs": _table(0, 65536, ROPE // 2), "ring": RING if case["ring"] else 0,
            "w": (1 + 0.2 * _randn(g, DIM)) if case["norm"] else None}


def _shape_of(case):
    """Compressed entries and drafted tokens of each sequence, by the case alone."""
    B, N, nodes = case["seqs"], case.get("N", 512), case["nodes"]
    if case["fill"] == "full":
        return [(N, nodes)] * B
    return [(int(N * ((b + 0.5) / B) ** 2), 0 if b == 0 and B > 1 else 1 + b * 7919 % nodes) for b in range(B)]


def _trees(case, seed):
    """Committed tokens and drafted tokens of a batch: a sequence's first node, positions, ancestors."""
    rnd = np.random.RandomState(int(seed) % (2 ** 31) + 17)
    seqs = [_shape_of(case)[b] for b in rnd.permutation(case["seqs"])]
    start, ctx, pos, anc = [0], [], [], []
    for entries, nodes in seqs:
        c = entries * 128 + int(rnd.randint(0, 128))
        ctx.append(c)
        depth, mask = [], []
        for j in range(nodes):
            p = j - 1 if case["shape"] == "chain" else max(-1, j - 1 - int(rnd.randint(0, 4)))
            depth.append(depth[p] + 1 if p >= 0 else 0)
            mask.append((mask[p] if p >= 0 else 0) | 1 << j)
        pos += [c + d for d in depth]
        anc += mask
        start.append(start[-1] + nodes)
    pad = 3 if case["fill"] == "ragged" else 0           # rows behind the last sequence
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    n_vis = [min((p + 1) // 128, case.get("N", 512)) for p in pos]
    return {"seqs": seqs, "max_nodes": case["nodes"], "T": len(pos) + pad, "start": i32(start), "ctx": i32(ctx),
            "pos": i32(pos + [0] * pad), "n_vis": i32(n_vis + [0] * pad),
            "anc": torch.from_numpy(np.array(anc + [0] * pad, dtype=np.uint64).astype(np.int64)).to(DEV),
            "seq_row": i32(rnd.permutation(case["seqs"]).tolist())}


def _prepare_list(case, g, seed):
    s = _trees(case, seed)
    s["idx_w"] = torch.full((s["T"], WINDOW + case["nodes"]), -2, dtype=torch.int32, device=DEV)
    return s


def _prepare_tree(case, g, seed):
    B, H, N, kind = case["seqs"], case["H"], case["N"], case["kind"]
    s = _trees(case, seed)
    T = s["T"]
    per = -(-N // PAGE)
    win_per = (DRAFT + 64) // PAGE
    s.update({"kind": kind, "n_max": N, "q": _randn(g, T, H, DIM).to(torch.bfloat16), "sink": _randn(g, H),
              "comp": _random_pages(g, kind, B * per + 2), "comp_pt": _page_table(g, B, per, B * per + 2),
              "win": _random_pages(g, kind, B * win_per + 2), "win_pt": _page_table(g, B, win_per, B * win_per + 2),
              "out": torch.zeros(T, H, DIM, dtype=torch.bfloat16, device=DEV),
              "lse": torch.zeros(T, H, dtype=torch.float32, device=DEV)})
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return globals()[("_own_" if own else "_plain_") + s["op"]](s)


def _own_table(s):
    _lib().dsv4sa_rope_table(s["cs"], first=s["first"], **YARN)
    return {"cs": s["cs"]}


def _own_rope(s):
    L = _lib()
    L.dsv4sa_rope(s["x"], s["cs"], s["pos"], out=s["out"], layout=L.ROPE_HALVES if s["halves"] else L.ROPE_PAIRS,
                  eps=EPS if s["norm"] else None)
    return {"out": s["out"]}


def _pool_values(s):
    """The pool as the values its bytes stand for; 4-bit codes, two a byte, as the bytes."""
    codes, rope, scale = _blocks(s["pool"], s["kind"])
    if s["kind"] == "kv":
        return {"codes": codes.view(torch.float8_e4m3fn), "rope": rope.view(torch.bfloat16),
                "scale": scale.view(torch.float32)[..., :7]}
    return {"codes": codes, "rope": rope.view(torch.bfloat16), "scale": scale[..., :14]}


def _own_append(s):
    _lib().dsv4sa_cache_append(s["desc"], s["table"], s["row_seq"], s["row_pos"], s["rows"], s["cs"], ring=s["ring"],
                               norm_w=s["w"], eps=EPS if s["w"] is not None else None)
    return _pool_values(s)


def _own_list(s):
    _lib().dsv4sa_tree_window_indices(s["start"], s["ctx"], s["pos"], WINDOW, RING, DRAFT, s["max_nodes"], s["idx_w"], anc=s["anc"])
    return {"idx_w": s["idx_w"]}


def _own_tree(s):
    _lib().dsv4sa_tree_attn(s["q"], s["sink"], s["start"], s["ctx"], s["pos"], s["comp_desc"], s["comp_pt"], s["n_vis"], s["n_max"],
                            s["win_desc"], s["win_pt"], WINDOW, s["out"], SOFTMAX_SCALE, max_nodes=s["max_nodes"],
                            seq_row=s["seq_row"], anc=s["anc"], win_ring=RING, draft_entry=DRAFT, lse=s["lse"], ws=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], by its bits."""
    e = e.to(torch.int32)
    return torch.where(e == -127, 0x00400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(v, kind):
    """fp32 values [n, 448] -> (code bytes, scale bytes) of the pool's kind."""
    n = v.shape[0]
    if kind == "kv":
        blk = v.view(n, 7, 64)
        scale = blk.abs().amax(-1).clamp(min=1e-4) * torch.tensor(1.0 / 448.0, dtype=torch.float32, device=v.device)
        codes = (blk / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes.view(torch.uint8).view(n, NOPE), scale.view(torch.uint8)
    blk = v.view(n, 14, 32)
    amax = blk.abs().amax(-1).clamp(min=6.0 * 2.0 ** -126)
    m, e = torch.frexp(amax * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=v.device))   # m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)                                                        # ceil(log2)
    y = (blk * _pow2(-e)[..., None]).clamp(-6, 6)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).view(n, NOPE)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _dequantise(codes, rope, scale, kind):
    """Bytes of rows -> fp32 values [..., 512], the nope part rounded to BF16 as the attention reads it."""
    if kind == "kv":
        v = codes.view(torch.float8_e4m3fn).float()
        f = scale.contiguous().view(torch.float32)[..., :7].repeat_interleave(64, dim=-1)
    else:
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=codes.device)
        v = lut[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()]
        f = _pow2(scale[..., :14].to(torch.int32) - 127).repeat_interleave(32, dim=-1)
    return torch.cat(((v * f).to(torch.bfloat16).float(), rope.contiguous().view(torch.bfloat16).float()), dim=-1)


def _rotate(x, cs, halves):
    """Pairs of the last dim of x [..., d] turned by cs [..., d / 2, 2]."""
    c, s = cs[..., 0], cs[..., 1]
    if halves:
        a, b = x.chunk(2, dim=-1)
        return torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)


def _plain_table(s):
    rows, pairs = s["cs"].shape[:2]
    s["cs"].copy_(_table(s["first"], rows, pairs))
    return {"cs": s["cs"]}


def _plain_rope(s):
    T, H, dim = s["x"].shape
    step = max(1, 2 ** 26 // (H * dim))
    for a in range(0, T, step):
        x = s["x"][a:a + step].float()
        if s["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        cs = s["cs"][s["pos"][a:a + step].long()][:, None]
        s["out"][a:a + step, :, :dim - s["rope"]] = x[..., :dim - s["rope"]].to(torch.bfloat16)
        s["out"][a:a + step, :, dim - s["rope"]:] = _rotate(x[..., dim - s["rope"]:], cs, s["halves"]).to(torch.bfloat16)
    return {"out": s["out"]}


def _slots(table, seq, entry):
    e = entry.long().clamp(min=0)
    return table[seq.long(), e // PAGE].long(), e % PAGE


def _plain_append(s):
    x = s["rows"].float()
    if s["w"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    c, sc = _quantise(x[:, :NOPE], s["kind"])
    r = _rotate(x[:, NOPE:], s["cs"][s["row_pos"].long()], False).to(torch.bfloat16)
    codes, rope, scale = _blocks(s["pool"], s["kind"])
    page, slot = _slots(s["table"], s["row_seq"], s["row_pos"] % s["ring"] if s["ring"] else s["row_pos"])
    codes[page, slot] = c
    rope[page, slot] = r.view(torch.uint8)
    scale[..., :sc.shape[-1]][page, slot] = sc
    return _pool_values(s)


def _gather(s, name, row, entry):
    codes, rope, scale = _blocks(s[name], s["kind"])
    page, slot = _slots(s[name + "_pt"], row, entry)
    return _dequantise(codes[page, slot], rope[page, slot], scale[page, slot], s["kind"])


def _attend(s, a, b, kv, ok):
    """Nodes a .. b over rows kv [r, 512] where ok [b - a, r]."""
    x = torch.matmul(s["q"][a:b].float(), kv.T) * SOFTMAX_SCALE
    x = x.masked_fill(~ok[:, None, :], -math.inf)
    m = torch.maximum(x.amax(-1), s["sink"][None])
    p = torch.exp(x - m[..., None])
    z = p.sum(-1) + torch.exp(s["sink"][None] - m)
    s["out"][a:b] = (torch.matmul(p, kv) / z[..., None]).to(torch.bfloat16)
    s["lse"][a:b] = m + torch.log(z)


def _plain_list(s):
    n = sum(n for _, n in s["seqs"])
    seq = torch.searchsorted(s["start"].long(), torch.arange(n, device=DEV), right=True) - 1
    j = torch.arange(s["max_nodes"], device=DEV)
    pos, ctx = s["pos"][:n, None].long(), s["ctx"].long()[seq][:, None]
    p = pos - WINDOW + 1 + torch.arange(WINDOW, device=DEV)
    seen = ((s["anc"][:n, None] >> j) & 1 == 1) & (j < (s["start"][1:] - s["start"][:-1])[seq][:, None])
    s["idx_w"][:n, :WINDOW] = torch.where((p >= 0) & (p < ctx), p % RING, -1)
    s["idx_w"][:n, WINDOW:] = torch.where(seen, DRAFT + j, -1)
    return {"idx_w": s["idx_w"]}


def _plain_tree(s):
    H = s["q"].shape[1]
    a = 0
    bits = torch.arange(64, device=DEV)
    for i, (_, nodes) in enumerate(s["seqs"]):
        if nodes == 0:
            continue
        row, ctx = s["seq_row"][i], s["ctx"][i]
        pos, n_vis = s["pos"][a:a + nodes, None], s["n_vis"][a:a + nodes, None]
        p = ctx - WINDOW + torch.arange(WINDOW, device=DEV)
        win = _gather(s, "win", row.expand(WINDOW), torch.where(p >= 0, p % RING, 0))
        drafts = _gather(s, "win", row.expand(nodes), DRAFT + bits[:nodes])
        e = torch.arange(s["n_max"], device=DEV)
        kv = torch.cat((_gather(s, "comp", row.expand(e.shape[0]), e), win, drafts))
        ok = torch.cat((e < n_vis, (p >= 0) & (p > pos - WINDOW) & (p <= pos), (s["anc"][a:a + nodes, None] >> bits[:nodes]) & 1 == 1), 1)
        step = max(1, 2 ** 28 // (H * kv.shape[0]))
        for j in range(0, nodes, step):
            _attend(s, a + j, a + min(nodes, j + step), kv, ok[j:j + step])
        a += nodes
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] == "list":
        return None          # whole numbers
    s = globals()["_prepare_" + case["op"]](case, _gen(seed), seed)
    return globals()["_exact_" + case["op"]](case, s)


def _turned(v, turns, halves):
    """v [..., 2 m] (fp64) as complex numbers times unit complex numbers [..., m]."""
    m = v.shape[-1] // 2
    z = torch.complex(v[..., :m].contiguous(), v[..., m:].contiguous()) if halves else torch.view_as_complex(v.reshape(*v.shape[:-1], m, 2))
    z = z * turns
    return torch.cat((z.real, z.imag), -1) if halves else torch.view_as_real(z).flatten(-2)


def _exact_table(case, s):
    rows, pairs = case["rows"], case["pairs"]
    y = YARN
    i = torch.arange(pairs, dtype=torch.float64, device=DEV)
    w = torch.exp(-(i / pairs) * math.log(y["base"]))
    border = lambda beta: 2 * pairs * math.log(y["original_len"] / (2 * math.pi * beta)) / (2 * math.log(y["base"]))  # noqa: E731
    lo, hi = max(math.floor(border(y["beta_fast"])), 0), min(math.ceil(border(y["beta_slow"])), 2 * pairs - 1)
    slow = ((i - lo) / (hi - lo)).clamp(0, 1)
    turn = (w * (slow / y["factor"] + (1 - slow))) / (2 * math.pi)
    out = torch.empty(rows, pairs, 2, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 131072):
        b = min(rows, a + 131072)
        t = (s["first"] + torch.arange(a, b, device=DEV, dtype=torch.float64))[:, None] * turn
        t = (t - torch.round(t)) * (2 * math.pi)
        out[a:b] = torch.view_as_real(torch.polar(torch.ones_like(t), t))
    return {"cs": out}


def _exact_rope(case, s):
    T, H, dim = s["x"].shape
    keep = dim - case["rope"]
    out = torch.empty(T, H, dim, dtype=torch.float64, device=DEV)
    turns = torch.view_as_complex(s["cs"].double())
    step = max(1, 2 ** 24 // (H * dim))
    for a in range(0, T, step):
        x = s["x"][a:a + step].double()
        if case["norm"]:
            x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / dim + EPS)
        out[a:a + step, :, :keep] = x[..., :keep]
        out[a:a + step, :, keep:] = _turned(x[..., keep:], turns[s["pos"][a:a + step].long()][:, None], case["halves"])
    return {"out": out}


def _e4m3(v):
    """fp64 -> the nearest E4M3 value, ties to even, as fp64."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    q = torch.exp2(e - 3)
    return (torch.round(v / q) * q).clamp(-448, 448)


def _exact_append(case, s):
    kind = case["kind"]
    pages = s["pool"].shape[0]
    x = s["rows"].double()
    if s["w"] is not None:
        x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / DIM + EPS) * s["w"].double()
    entry = s["row_pos"].long()
    if s["ring"]:
        entry = entry % s["ring"]
    at = s["table"].long()[s["row_seq"].long(), entry // PAGE] * PAGE + entry % PAGE
    rope = torch.zeros(pages * PAGE, ROPE, dtype=torch.float64, device=DEV)
    rope[at] = _turned(x[:, NOPE:].contiguous(), torch.view_as_complex(s["cs"].double())[s["row_pos"].long()], False)
    out = {"codes": None, "rope": rope.view(pages, PAGE, ROPE), "scale": None}      # 4-bit codes and exponents: whole numbers
    if kind == "kv":
        blk = x[:, :NOPE].reshape(-1, 7, 64)
        top = blk.abs().amax(-1).clamp(min=1e-4) / 448.0
        codes = torch.zeros(pages * PAGE, NOPE, dtype=torch.float64, device=DEV)
        scale = torch.zeros(pages * PAGE, 7, dtype=torch.float64, device=DEV)
        codes[at] = _e4m3(blk / top[..., None]).view(-1, NOPE)
        scale[at] = top
        out["codes"], out["scale"] = codes.view(pages, PAGE, NOPE), scale.view(pages, PAGE, 7)
    return out


def _values(s, name):
    """Every slot of a pool in fp64 [pages * 64, 512], the nope part rounded to BF16 as the cache is read."""
    codes, rope, scale = _blocks(s[name], s["kind"])
    P = s[name].shape[0]
    if s["kind"] == "kv":
        byte = codes.int()
        e, m = (byte >> 3) & 15, byte & 7
        mag = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * torch.exp2((e - 10).double()))
        v = torch.where(byte >= 128, -mag, mag).view(P, PAGE, 7, 64) * scale.contiguous().view(torch.float32)[..., :7, None].double()
    else:
        nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[nib % 8]
        v = torch.where(nib >= 8, -mag, mag).view(P, PAGE, 14, 32) * torch.exp2(scale[..., :14, None].double() - 127)
    out = torch.empty(P * PAGE, DIM, dtype=torch.float64, device=DEV)
    # products of at most 28 significant bits: by way of fp32 the BF16 rounding may differ at a tie's neighbour only
    out[:, :NOPE] = v.reshape(-1, NOPE).float().to(torch.bfloat16)
    out[:, NOPE:] = rope.contiguous().view(torch.bfloat16).view(-1, ROPE)
    return out


def _exact_tree(case, s):
    T, H = s["q"].shape[:2]
    comp, win = _values(s, "comp"), _values(s, "win")
    out = torch.zeros(T, H, DIM, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    start, ctx, pos = s["start"].tolist(), s["ctx"].tolist(), s["pos"].tolist()
    n_vis, anc, row = s["n_vis"].tolist(), s["anc"].tolist(), s["seq_row"].tolist()
    for b in range(len(start) - 1):
        comp_at = (s["comp_pt"][row[b]].long()[:, None] * PAGE + torch.arange(PAGE, device=DEV)).view(-1)
        win_at = (s["win_pt"][row[b]].long()[:, None] * PAGE + torch.arange(PAGE, device=DEV)).view(-1)
        for t in range(start[b], start[b + 1]):
            slots = [p % RING for p in range(max(0, pos[t] - WINDOW + 1), min(pos[t] + 1, ctx[b]))]
            slots += [DRAFT + j for j in range(start[b + 1] - start[b]) if anc[t] >> j & 1]
            rows = torch.cat((comp[comp_at[:n_vis[t]]], win[win_at[torch.tensor(slots, dtype=torch.long, device=DEV)]]))
            x = torch.cat((s["q"][t].double() @ rows.T * SOFTMAX_SCALE, s["sink"].double()[:, None]), 1)
            z = torch.logsumexp(x, -1)
            out[t], lse[t] = torch.exp(x[:, :-1] - z[:, None]) @ rows, z
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": case["rows"] * case["pairs"] * 8, "flops": 2 * case["rows"] * case["pairs"]}
    if op == "rope":
        T, H, dim = case["T"], case["H"], case["dim"]
        return {"bytes": T * H * dim * 4 + T * (case["rope"] * 4 + 4), "flops": T * H * (3 * case["rope"] + (3 * dim if case["norm"] else 0))}
    if op == "append":
        # each BF16 row and its rotation read, the packed row written
        per = 1024 + 256 + 8 + ROW_BYTES[case["kind"]]
        return {"bytes": case["n"] * per + (2048 if case["norm"] else 0), "flops": case["n"] * DIM * (6 if case["norm"] else 3)}
    if op == "list":
        T = sum(nodes for _, nodes in _shape_of(case))
        return {"bytes": T * (12 + 4 * (WINDOW + case["nodes"])) + case["seqs"] * 8, "flops": 0}
    H = case["H"]
    nbytes = flops = 0
    for entries, nodes in _shape_of(case):
        if nodes == 0:
            continue
        window = min(WINDOW, entries * 128 + 64)
        # a sequence's rows once; each node's queries and outputs
        nbytes += (entries + window + nodes) * ROW_BYTES[case["kind"]] + nodes * H * (2048 + 4) + nodes * 16
        flops += 4 * DIM * H * nodes * (entries + window)
    return {"bytes": nbytes, "flops": flops}
