"""Strides of rotated heads that no memory spans: refused, for any number of tokens and heads."""
import ctypes

import pytest

from test_cache_norm_cpu import INVALID, ptr
from test_drafts_cpu import L, rope_args  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(T=2 ** 25 + 1, H=8, out_tok_stride=2 ** 39, x_tok_stride=4096),
    dict(T=2 ** 25 + 1, H=8, x_tok_stride=2 ** 39),                        # 2^64 values: the span was that of one token
    dict(T=2 ** 29, H=1, x_tok_stride=2 ** 40),
    dict(T=1, H=2 ** 25 + 1, x_head_stride=2 ** 39, out_head_stride=512),
    dict(T=1, H=2 ** 25 + 1, out_head_stride=2 ** 39, x_head_stride=512),
    dict(T=2 ** 22, H=8, x_tok_stride=2 ** 20)])
def test_spans_past_any_memory(L, kw):
    a = rope_args(L, **{**dict(out=ptr(2 ** 30), rope_cs=ptr(2 ** 29), pos=ptr(2 ** 28), norm_w=None, x=ptr(2 ** 32)), **kw})
    assert L.lib().dsv4sa_rope(ctypes.byref(a), None) == INVALID
