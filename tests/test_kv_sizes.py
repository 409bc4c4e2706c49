"""Sizes at which the host's choices have to hold, without a GPU."""

import pytest

pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")


def workspace(tokens=64, heads=32, kv=2, dim=128, block=64, width=128, requests=64, max_new=1, max_context=8192, window=0):
    return qw.library().qw_kv_attention_workspace(tokens, heads, kv, dim, block, width, requests, max_new, max_context, window)


def test_ranges_only_where_their_sums_fit():
    """The device sums 64-key tiles over all units in int32.  Without a causal
    mask, and with more queries than max_new, a window bounds none of them: where
    2^21 tiles of 1500 units could pass 2^31, there are no ranges."""
    sizes = dict(tokens=48000, heads=1, kv=1, dim=64, width=1 << 21, requests=1, max_new=48000)
    assert workspace(max_context=1 << 27, window=64, **sizes) == 0
    assert workspace(max_context=1 << 27, **sizes) == 0
    assert workspace(max_context=1 << 26, window=64, **sizes) > 0
