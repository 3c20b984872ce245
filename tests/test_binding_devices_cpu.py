"""Every tensor and pool of a call has to be on the current device.  No second GPU is needed:
the tensors here are host tensors that say which device they are on, and the library's
entry points only count that they were reached."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


class On(torch.Tensor):
    """A host tensor that passes for one of cuda:`gpu`."""
    gpu = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.gpu


def on(shape, dtype, gpu=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.gpu = gpu
    return t


i32, f32, u8, bf16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16


def calls(L):
    """name -> (tensors by name: (shape, dtype), pool kinds by name, the call)."""
    attn_t = dict(q=((2, 16, 512), bf16), attn_sink=((16,), f32), q_seq=((2,), i32), comp_pt=((2, 4), i32), idx_c=((2, 8), i32),
                  win_pt=((2, 4), i32), out=((2, 16, 512), bf16), lse=((2, 16), f32), ws=((64,), u8), rope_cs=((5, 32, 2), f32),
                  rope_pos=((2,), i32))
    both = dict(comp=L.POOL_KV_FP4, win=L.POOL_KV_FP4)

    def attn(fn, *first):
        def go(t, p):
            idx_w, pos = t.get("idx_w"), t.get("win_pos")
            kw = dict(win_pos=pos, kw=16) if pos is not None else {}
            if first:
                kw["topk_ws"] = t["topk_ws"]
            lead = (t["logits"], t["n_vis"], 8, 8) if first else ()
            fn(*lead, t["q"], t["attn_sink"], t["q_seq"], p["comp"], t["comp_pt"], t["idx_c"], p["win"], t["win_pt"], idx_w, t["out"],
               0.04, lse=t["lse"], ws=t["ws"], rope_cs=t["rope_cs"], rope_pos=t["rope_pos"], **kw)
        return go
    lists = dict(idx_w=((2, 16), i32))
    positions = dict(win_pos=((2,), i32))
    rows = dict(page_table=((2, 4), i32), row_seq=((3,), i32), row_entry=((3,), i32))
    idx = dict(page_table=((2, 4), i32), q_seq=((2,), i32), n_vis=((2,), i32), w=((2, 4), f32), logits=((2, 8), f32))
    topk = dict(logits=((2, 8), f32), n_vis=((2,), i32), idx=((2, 8), i32), ws=((64,), u8))
    c128 = dict(kv=((3, 512), bf16), score=((3, 512), bf16), state_idx=((3,), i32), state=((4, 3, 512), f32), state_count=((4,), i32),
                position=((3,), i32), ape=((128, 512), f32), norm_w=((512,), f32), rope_cs=((5, 32, 2), f32), out=((3, 512), bf16),
                done=((3,), i32))
    win = dict(kv=((8, 1024), bf16), score=((8, 1024), bf16), first_tok=((2,), i32), prev_tok=((2,), i32), position=((2,), i32),
               ape=((4, 1024), f32), norm_w=((512,), f32), rope_cs=((5, 32, 2), f32), out=((2, 512), bf16))
    key = dict(kpool=L.POOL_IDXK)
    return {
        "indexer_logits": ({**idx, "q_fp8": ((2, 4, 128), u8), "q_scale": ((2, 4, 2), f32)}, key, lambda t, p: L.dsv4sa_indexer_logits(
            p["kpool"], t["page_table"], t["q_seq"], t["n_vis"], t["q_fp8"], t["q_scale"], t["w"], 8, t["logits"])),
        "indexer_logits_fp4": ({**idx, "q_fp4": ((2, 4, 64), u8), "q_e8m0": ((2, 4, 4), u8)}, key, lambda t, p: L.dsv4sa_indexer_logits_fp4(
            p["kpool"], t["page_table"], t["q_seq"], t["n_vis"], t["q_fp4"], t["q_e8m0"], t["w"], 8, t["logits"])),
        "topk": (topk, {}, lambda t, p: L.dsv4sa_topk(t["logits"], t["n_vis"], 8, 8, t["idx"], t["ws"])),
        "topk_noalloc": ({k: topk[k] for k in ("logits", "n_vis", "idx")}, {}, lambda t, p: L.dsv4sa_topk_noalloc(
            t["logits"], t["n_vis"], 8, 8, t["idx"])),
        "topk_prefetch": ({**topk, "kv_pt": ((2, 4), i32), "q_seq": ((2,), i32)}, dict(kv_pool=L.POOL_KV), lambda t, p: L.dsv4sa_topk_prefetch(
            t["logits"], t["n_vis"], 8, 8, t["idx"], p["kv_pool"], t["kv_pt"], t["q_seq"], t["ws"])),
        "window_indices": (dict(pos=((2,), i32), idx_w=((2, 8), i32)), {}, lambda t, p: L.dsv4sa_window_indices(t["pos"], 8, 0, t["idx_w"])),
        "compress_indices": (dict(n_vis=((2,), i32), idx=((2, 8), i32)), {}, lambda t, p: L.dsv4sa_compress_indices(t["n_vis"], 8, t["idx"])),
        "cache_write": ({**rows, "rows": ((3, 512), bf16)}, dict(pool=L.POOL_KV_FP4), lambda t, p: L.dsv4sa_cache_write(
            p["pool"], t["page_table"], t["row_seq"], t["row_entry"], t["rows"])),
        "cache_write_rotated": ({**rows, "rows": ((3, 128), bf16)}, dict(pool=L.POOL_IDXK_FP4), lambda t, p: L.dsv4sa_cache_write_rotated(
            p["pool"], t["page_table"], t["row_seq"], t["row_entry"], t["rows"])),
        "cache_read": ({**rows, "rows": ((3, 512), bf16)}, dict(pool=L.POOL_KV_FP4), lambda t, p: L.dsv4sa_cache_read(
            p["pool"], t["page_table"], t["row_seq"], t["row_entry"], t["rows"])),
        "pages_copy": (dict(src_page=((3,), i32), dst_page=((3,), i32)), dict(pool=L.POOL_KV), lambda t, p: L.dsv4sa_pages_copy(
            [p["pool"]], t["src_page"], t["dst_page"])),
        "page_cache": (dict(page_table=((2, 4), i32), use=((4,), i32)), dict(pool=L.POOL_KV), lambda t, p: (
            L.page_cache([p["pool"]], t["page_table"], t["use"]), L.lib().reached())),
        "rmsnorm_quant": (dict(x=((4, 256), bf16), norm_w=((256,), f32), codes=((4, 256), u8), scale=((4, 2), f32), residual=((4, 256), bf16),
                               residual_out=((4, 256), bf16), y=((4, 256), bf16)), {}, lambda t, p: L.dsv4sa_rmsnorm_quant(
            t["x"], t["norm_w"], t["codes"], t["scale"], residual=t["residual"], residual_out=t["residual_out"], y=t["y"])),
        "compress_windows": (win, {}, lambda t, p: L.dsv4sa_compress_windows(
            t["kv"], t["score"], t["first_tok"], t["prev_tok"], t["position"], 4, True, t["ape"], t["norm_w"], t["rope_cs"], t["out"])),
        "compress_online_c128": (c128, {}, lambda t, p: L.dsv4sa_compress_online_c128(
            t["kv"], t["score"], t["state_idx"], t["state"], t["state_count"], t["position"], t["ape"], t["norm_w"], t["rope_cs"], t["out"],
            t["done"])),
        "selftest_wait_timeout": (dict(result=((1,), i32)), {}, lambda t, p: L.dsv4sa_selftest_wait_timeout(t["result"])),
        "copy_async": (dict(dst=((16,), u8), src=((16,), u8)), {}, lambda t, p: L.dsv4sa_copy_async(t["dst"], t["src"])),
        "copy_async_background": (dict(dst=((16,), u8), src=((16,), u8)), {}, lambda t, p: L.dsv4sa_copy_async_background(t["dst"], t["src"])),
        "sparse_attn_decode": ({**attn_t, **lists}, both, attn(L.dsv4sa_sparse_attn_decode)),
        "sparse_attn_prefill": ({**attn_t, **positions}, both, attn(L.dsv4sa_sparse_attn_prefill)),
        "topk_sparse_attn_decode": ({**attn_t, **positions, "logits": ((2, 8), f32), "n_vis": ((2,), i32), "topk_ws": ((64,), u8)}, both,
                                    attn(L.dsv4sa_topk_sparse_attn_decode, True)),
    }


NAMES = ["indexer_logits", "indexer_logits_fp4", "topk", "topk_noalloc", "topk_prefetch", "window_indices", "compress_indices", "cache_write",
         "cache_write_rotated", "cache_read", "pages_copy", "page_cache", "rmsnorm_quant", "compress_windows", "compress_online_c128",
         "selftest_wait_timeout", "copy_async", "copy_async_background", "sparse_attn_decode", "sparse_attn_prefill",
         "topk_sparse_attn_decode"]


class Reached:
    """Stands in for the library: every entry point succeeds and is counted."""

    def __init__(self, real):
        self.real, self.n = real, 0

    def reached(self):
        self.n += 1

    def __getattr__(self, name):
        def fn(*a):
            self.n += 1
            return 0
        return fn if name.startswith("dsv4sa") and name != "dsv4sa_pool_desc_init" else getattr(self.real, name)


@pytest.fixture
def stub(L, monkeypatch):
    s = Reached(L.lib())
    monkeypatch.setattr(L, "lib", lambda: s)
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda d: 0)
    return s


def pool(L, kind, gpu=0):
    nbytes = 4 * 38912
    buf = on((nbytes + 1024,), u8, gpu)
    base = buf[-buf.data_ptr() % 1024:]
    base.gpu = gpu
    return L.dsv4sa_pool_desc_init(kind, base, 4)


@pytest.mark.parametrize("name", NAMES)
def test_each_tensor_and_pool_is_checked(L, stub, name):
    tensors, pools, go = calls(L)[name]

    def run(away=None):
        go({k: on(s, d, int(k == away)) for k, (s, d) in tensors.items()}, {k: pool(L, kind, int(k == away)) for k, kind in pools.items()})
    run()
    assert stub.n == 1                                            # all of them at home: the library is called
    for k in [*tensors, *pools]:
        with pytest.raises(ValueError, match=f"^{k} is on cuda:1, the current device is cuda:0$"):
            run(k)
    assert stub.n == 1


def test_names_are_all_there(L):
    assert sorted(calls(L)) == sorted(NAMES)


def test_caches_are_checked_when_they_are_used(L, stub, monkeypatch):
    """A cache made on one device, used while another one is current (its lists on that one)."""
    def make(gpu):
        monkeypatch.setattr(L, "_current_device", lambda: gpu)
        c = L.page_cache([pool(L, L.POOL_KV, gpu)], on((2, 4), i32, gpu), on((4,), i32, gpu))
        monkeypatch.setattr(L, "_current_device", lambda: 0)
        return c
    here, away = make(0), make(1)
    r, ids, one = on((2,), i32), on((4,), i32), on((1,), i32)
    L.dsv4sa_cache_release(here, r)
    L.dsv4sa_cache_fork(here, r, r, r, r)
    L.dsv4sa_cache_compact(here, here, ids, one)
    assert stub.n == 3
    for call, word in ((lambda: L.dsv4sa_cache_release(away, r), "cache"), (lambda: L.dsv4sa_cache_fork(away, r, r, r, r), "cache"),
                       (lambda: L.dsv4sa_cache_compact(away, here, ids, one), "src"),
                       (lambda: L.dsv4sa_cache_compact(here, away, ids, one), "dst")):
        with pytest.raises(ValueError, match=f"^{word} is on cuda:1"):
            call()
    far = on((2,), i32, 1)
    for args in ((far, r, r, r), (r, far, r, r), (r, r, far, r), (r, r, r, far)):
        with pytest.raises(ValueError, match="is on cuda:1"):
            L.dsv4sa_cache_fork(here, *args)
    for call in (lambda: L.dsv4sa_cache_release(here, far), lambda: L.dsv4sa_cache_compact(here, here, on((4,), i32, 1), one),
                 lambda: L.dsv4sa_cache_compact(here, here, ids, on((1,), i32, 1))):
        with pytest.raises(ValueError, match="is on cuda:1"):
            call()
    assert stub.n == 3


def test_pools_of_addresses_and_host_memory_have_no_device_to_compare(L, stub):
    rows = [on(s, d) for s, d in (((2, 4), i32), ((3,), i32), ((3,), i32), ((3, 512), bf16))]
    host = torch.zeros(4 * 23552 + 1024, dtype=u8)
    for base in (1 << 20, host[-host.data_ptr() % 1024:]):
        L.dsv4sa_cache_write(L.dsv4sa_pool_desc_init(L.POOL_KV_FP4, base, 4), *rows)
    assert stub.n == 2
