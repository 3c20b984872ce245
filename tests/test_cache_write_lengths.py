"""The cache writers read row_seq[r] and row_entry[r] for every row: shorter lists are refused."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_c4_gb300 import build, dsv4sa
    if not os.path.exists(dsv4sa.LIB_PATH):
        build.build()
    return dsv4sa


@pytest.mark.parametrize("writer,kind,width", [("dsv4sa_cache_write", 0, 512), ("dsv4sa_cache_write", 1, 128), ("dsv4sa_cache_write", 2, 128),
                                               ("dsv4sa_cache_write", 3, 512), ("dsv4sa_cache_write_rotated", 2, 128)])
def test_lists_shorter_than_the_rows_are_refused(L, writer, kind, width):
    pool = L.dsv4sa_pool_desc_init(kind, 1 << 20, 4)
    i32, rows = torch.zeros(6, dtype=torch.int32), torch.zeros(5, width, dtype=torch.bfloat16)
    for seq, entry in ((i32[:4], i32[:5]), (i32[:5], i32[:4]), (i32[:0], i32[:5]), (i32[:5], i32[:0])):
        with pytest.raises(ValueError, match="one entry for each of the 5 rows"):
            getattr(L, writer)(pool, i32[None], seq, entry, rows)
    for n in (5, 6):                                             # enough: the call goes on to the tensors' devices
        with pytest.raises(ValueError, match="CUDA tensor"):
            getattr(L, writer)(pool, i32[None], i32[:n], i32[:n], rows)


@pytest.mark.gpu
def test_longer_lists_write_the_rows_there_are(L):
    bufs = [L._alloc_pool(L.POOL_KV_FP4, 2, "cuda").zero_() for _ in range(2)]
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    entry = torch.tensor([3, 64, 7, 100], dtype=torch.int32, device="cuda")
    rows = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    for buf, n in zip(bufs, (3, 4)):
        L.dsv4sa_cache_write(L.dsv4sa_pool_desc_init(L.POOL_KV_FP4, buf, 2), table, torch.zeros_like(entry[:n]), entry[:n].clone(), rows)
    assert L.dsv4sa_check_errors() == (0, 0) and torch.equal(*bufs) and bool(bufs[0].any())
