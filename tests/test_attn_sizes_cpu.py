"""The attention's binding refuses tensors that are too small for the queries of the call (the
kernel would read and write past their ends).  Host tensors that pass for device ones."""
import pytest

from test_binding_devices_cpu import L, bf16, f32, i32, on, pool, stub  # noqa: F401  (fixtures)

T, H, KC, KW = 5, 24, 40, 16
FULL = dict(attn_sink=(H,), q_seq=(T,), idx_c=(T, KC), idx_w=(T, KW), win_pos=(T,), out=(T, H, 512), lse=(T, H), rope_pos=(T,))
DTYPE = dict(attn_sink=f32, out=bf16, lse=f32)


def call(L, fn, explicit, **small):
    t = {k: on(small.get(k, s), DTYPE.get(k, i32)) for k, s in FULL.items()}
    pools = [pool(L, L.POOL_KV_FP4) for _ in range(2)]
    pt = on((3, 4), i32)
    window = dict(win_pos=None, kw=None) if explicit else dict(win_pos=t["win_pos"], kw=KW)
    fn(on((T, H, 512), bf16), t["attn_sink"], t["q_seq"], pools[0], pt, t["idx_c"], pools[1], pt, t["idx_w"] if explicit else None, t["out"],
       0.04, lse=t["lse"], rope_cs=on((9, 32, 2), f32), rope_pos=t["rope_pos"], **window)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_tensors_too_small_for_the_queries(L, stub, mode):  # noqa: F811
    fn = getattr(L, "dsv4sa_sparse_attn_" + mode)
    small = dict(attn_sink=(H - 1,), q_seq=(T - 1,), idx_c=(T - 1, KC), out=(T, H - 1, 512), lse=(T - 1, H), rope_pos=(T - 1,))
    for explicit, more in ((True, dict(idx_w=(T - 1, KW))), (False, dict(win_pos=(T - 1,)))):
        before = stub.n
        call(L, fn, explicit)
        call(L, fn, explicit, q_seq=(T + 3,), out=(T, H * 512), lse=(T * H,), attn_sink=(128,))   # other shapes, large enough
        assert stub.n == before + 2
        for k, s in {**small, **more}.items():
            with pytest.raises(ValueError, match=k):
                call(L, fn, explicit, **{k: s})
        assert stub.n == before + 2
