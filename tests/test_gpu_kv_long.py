"""kv_attention over prompts with more than 2^20 query rows."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import F16, dev, host, ints, unit, within  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,dim", [(64, 8, 128), (64, 8, 64)])
def test_prompt_of_many_rows(heads, kv, dim):
    rng = np.random.default_rng(dim)
    tokens, block = 32768, 64
    context = [tokens]
    table, blocks = ref.pages(rng, context, block)
    cache = ref.random_cache(rng, blocks, kv, dim, block)
    gen = torch.Generator(device="cuda:0").manual_seed(dim)
    q = torch.randn((tokens, heads, dim), generator=gen, device="cuda:0").to(F16)
    say("attention of %d tokens, %d/%d D=%d" % (tokens, heads, kv, dim))
    got = qw.kv_attention(q, *[dev(c) for c in cache], ints(table), ints(context), ints([0, tokens]), tokens)
    assert not torch.isnan(got).any()
    for at in (0, 1, 63, 64, 16383, 20000, tokens - 1):
        row = host(q[at:at + 1])
        want, mass, reach, tail = ref.attention_rows(row, cache, table, [at + 1], [0, 1], 1, dim ** -0.5)
        within(host(got[at:at + 1]), want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(F16)), "token %d" % at)
