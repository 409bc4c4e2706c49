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


def test_long_prompts_of_many_heads():
    """A prompt of 32768 tokens with 64 heads, one of 65536 with 32 and one of
    2^17 with 64 are taken, and a loose bound of the new tokens counts no more
    than the tokens of the call; beyond 2^23 rows a request they are refused."""
    def takes(tokens, max_new, heads):
        n = workspace(tokens=tokens, heads=heads, kv=8, width=1 << 14, requests=2, max_new=max_new, max_context=1 << 20)
        assert n >= -1
        return n >= 0
    assert takes(32768, 32768, 64) and takes(65536, 65536, 32) and takes(1 << 17, 1 << 17, 64)
    assert takes(64, 1 << 20, 64)
    assert not takes((1 << 17) + 1, (1 << 17) + 1, 64) and not takes(64, (1 << 20) + 1, 64)
