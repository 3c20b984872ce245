"""Which kernels the FP4 attention chooses for the batches that the parity tests run: heads of
an item, CTAs of a cluster, items a CTA -- read off the launches, captured and not run."""
import ctypes
import os

import pytest
import torch

from test_gpu_fp4_serving import test_every_split_of_heads_and_rows as parity_of_splits
from test_gpu_kv_fp4 import Case
from test_gpu_kv_fp4 import test_attention_matches_fp64 as parity_of_shapes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


class KernelNode(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """(name, CTAs, CTAs of a cluster) of every kernel that call(stream) launches, by a capture."""
    cu = ctypes.CDLL("libcuda.so.1")

    def do(fn, *a):
        assert getattr(cu, fn)(*a) == 0, fn
    stream, graph, n = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t()
    handle = ctypes.c_void_p(stream.cuda_stream)
    torch.cuda.synchronize()
    do("cuStreamBeginCapture_v2", handle, 2)
    try:
        call(stream)
    finally:
        do("cuStreamEndCapture", handle, ctypes.byref(graph))
    do("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    do("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    out = []
    for node in nodes:
        p, name, attr = KernelNode(), ctypes.c_char_p(), (ctypes.c_uint * 16)()
        do("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        if p.kern:
            do("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(p.kern))
        else:
            do("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(p.func))
        do("cuGraphKernelNodeGetAttribute", ctypes.c_void_p(node), 4, attr)       # the cluster's dimensions
        out.append((name.value.decode(), p.grid[0], max(1, attr[0])))
    do("cuGraphDestroy", graph)
    return out


def plan(L, T, H, kc, kw, mode="decode"):
    """(heads of an item, CTAs of a cluster, items a CTA at most)"""
    c = Case(L, T, H, min(kc, 64), kw, seed=1, ring=128)
    idx = torch.full((T, kc), -1, dtype=torch.int32, device="cuda")
    out, d = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), c.d
    fn = L.dsv4sa_sparse_attn_decode if mode == "decode" else L.dsv4sa_sparse_attn_prefill
    (name, ctas, cluster), = launches(lambda s: fn(d["q"], d["sink"], d["seq"], c.comp_d, d["comp_pt"], idx, c.win_d, d["win_pt"], None, out,
                                                   0.04, stream=s, win_pos=d["pos"], kw=kw, win_ring=128))
    heads = [h for h in (16, 32, 64) if f"sparse_attn_fp4_kernelILi{h}E" in name]
    assert len(heads) == 1, name
    items = T * -(-H // heads[0])
    assert ctas == items * cluster if cluster > 1 else ctas <= items
    return heads[0], cluster, -(-items * cluster // ctas)


def cases_of(test):
    """The sizes (T, H, kc, kw) that a parity test runs over."""
    sizes, = [m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0].startswith("T,H,kc")]
    return [(T, H, kc, *(rest[:1] or [128])) for T, H, kc, *rest in sizes if kc > 0]


def test_the_parity_cases_take_every_variant(L):
    """Items of 16, 32 and 64 heads, each as one CTA an item and over clusters; clusters of 2, 4
    and 8; several items a CTA.  (16 heads with one CTA an item take many queries of few heads,
    which test_attention_matches_fp64 has; the rest is in test_every_split_of_heads_and_rows.)"""
    plans = {c: plan(L, *c) for c in cases_of(parity_of_splits) + cases_of(parity_of_shapes)}
    print(plans)
    alone, split = {p[0] for p in plans.values() if p[1] == 1}, {p[0] for p in plans.values() if p[1] > 1}
    assert alone == split == {16, 32, 64}, plans
    assert {p[1] for p in plans.values()} == {1, 2, 4, 8}, plans
    assert any(p[2] > 1 for p in plans.values()), plans
    for c in cases_of(parity_of_splits):
        assert plan(L, *c, mode="prefill")[1] == 1                                  # prefill is never split
    assert L.dsv4sa_check_errors() == (0, 0)
