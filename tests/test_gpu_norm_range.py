"""The norm's quantised output at the ends of the fp32 range, and the operators' first calls
in a process made while a graph is captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from test_gpu_norm import bits, check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.mark.parametrize("dim,group", [(128, 64), (128, 128), (1024, 128), (4096, 64)])
@pytest.mark.parametrize("weight", [2e38, 9e37, 3e37, 1e-3, 1e-37])
def test_weights_of_any_size(L, dim, group, weight):
    """y = x w / rms with |w| from 1e-37 to 2e38 (x w stays in the fp32 range): the bounds of
    test_gpu_norm; a BF16 output is checked where it is finite."""
    g = torch.Generator().manual_seed(dim + group)
    x = (torch.randint(-5, 6, (9, dim), generator=g) / 4).to(torch.bfloat16).cuda()   # at most 1.25
    w = torch.full((dim,), weight, device="cuda")
    codes, scale = torch.empty(9, dim, dtype=torch.uint8, device="cuda"), torch.empty(9, dim // group, device="cuda")
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale, group=group, eps=1e-6)
    ref = oracle.rms_norm_quant(bits(x), None, w.cpu().numpy(), 1e-6, group)
    assert np.isfinite(ref["y"]).all() and np.abs(ref["y"]).max() < 3.4e38
    check(ref, codes=codes, scale=scale)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from compressed_sparse_attention_c4_gb300 import dsv4sa as L
torch.cuda.init()
T, H, P = 4, 64, 40
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
buf = L._alloc_pool(L.POOL_KV_FP4, P, "cuda"); buf.zero_()
pool = L.dsv4sa_pool_desc_init(L.POOL_KV_FP4, buf, P)
table = torch.full((6, 8), -1, dtype=torch.int32, device="cuda")
table[0] = torch.arange(8, dtype=torch.int32)
use = torch.zeros(P, dtype=torch.int32, device="cuda"); use[:8] = 1
cache = L.page_cache([pool], table, use)
n = 500
rows = torch.randn(n, 512, device="cuda").to(torch.bfloat16)
seq, ent = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
back = torch.zeros_like(rows)
q = torch.randn(T, H, 512, device="cuda").to(torch.bfloat16)
sink, qs = torch.zeros(H, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
idx = torch.randint(0, n, (T, 448), dtype=torch.int32, device="cuda")
out, out2 = torch.zeros_like(q), torch.zeros_like(q)
src, dst, ln, new = i32(0, 0), i32(1, 2), i32(100, 500), torch.zeros(2, dtype=torch.int32, device="cuda")
new_id, used = torch.zeros(P, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
x, w = torch.randn(8, 512, device="cuda").to(torch.bfloat16), torch.ones(512, device="cuda")
codes, scale = torch.zeros(8, 512, dtype=torch.uint8, device="cuda"), torch.zeros(8, 4, device="cuda")
def body():
    L.dsv4sa_cache_write(pool, table, seq, ent, rows)
    L.dsv4sa_cache_read(pool, table, seq, ent, back)
    L.dsv4sa_sparse_attn_decode(q, sink, qs, pool, table, idx, None, None, None, out, 0.04)
    L.dsv4sa_sparse_attn_prefill(q, sink, qs, pool, table, idx, None, None, None, out2, 0.04)
    L.dsv4sa_rmsnorm_quant(x, w, codes, scale)
    L.dsv4sa_cache_release(cache, i32_dst)
    L.dsv4sa_cache_fork(cache, src, dst, ln, new)
    L.dsv4sa_cache_compact(cache, cache, new_id, used)
i32_dst = i32(1, 2)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    body()
g.replay(); g.replay()
torch.cuda.synchronize()
assert L.dsv4sa_check_errors() == (0, 0)
got = [t.clone() for t in (back, out, out2, codes, scale, new, table, use, used)]
body()
torch.cuda.synchronize()
assert L.dsv4sa_check_errors() == (0, 0)
for a, b in zip(got, (back, out, out2, codes, scale, new, table, use, used)):
    assert torch.equal(a, b)
assert out.abs().max() > 0 and int(used) == 10, int(used)
print("done")
"""


def test_first_calls_of_a_process_while_capturing(L):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=250)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
