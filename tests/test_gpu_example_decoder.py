"""examples/decoder_attention.py: prompts and replayed decode steps through
all of the cache's operators between the two GEMMs."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [dict(hidden=256, heads=4, kv_heads=2, head_dim=64, requests=3, prompt=70, tokens=5),
                                   dict(hidden=512, heads=8, kv_heads=1, head_dim=128, requests=5, prompt=300, tokens=70)])
def test_decoder_attention(sizes):
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decoder_attention.py")
    spec = importlib.util.spec_from_file_location("decoder_attention", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error, _, _ = example.run(**sizes)
    # A value code is off by half a step, 1/254 of its block's largest, and a
    # key's likewise moves the scores by 1/254 of |q| |k| / sqrt(dim) at most;
    # with normed heads and keys within five deviations, independent errors
    # over the row leave some 2 % of an output's deviation.  An order of
    # magnitude less than what a wrong place, scale or position gives.
    assert error < 0.05
