"""examples/decoder_feed_forward.py: prompts and replayed decode steps through
all of the feed-forward operators."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decoder_feed_forward.py")
    spec = importlib.util.spec_from_file_location("decoder_feed_forward", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kind,tokens,prompt", [("dense", 3, 70), ("codes", 20, 300), ("experts", 1, 5), ("experts", 20, 300)])
def test_decoder_feed_forward(example, kind, tokens, prompt):
    layer = example.Experts(256, 128, 16, 4) if kind == "experts" else example.Dense(256, 512, kind == "codes")
    error, _, _ = example.run(layer, 256, tokens, prompt, steps=5)
    # fp16: each of three intermediate roundings is 2^-11 of its value, and the
    # last one too.  Codes: half a step, 1/254 of the row's largest, for each of
    # two products whose terms add up as independent errors: with largest
    # elements of four deviations 0.016 / sqrt(3) = 0.9 % of the output's
    # deviation each, against a largest output of four deviations.
    assert error < (0.03 if kind == "codes" else 0.005)
