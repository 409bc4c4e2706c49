"""kv_attention over requests whose numbers of new tokens differ: results, and
that one request with more of them does not make the others slow."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import F16, TYPES, ints  # noqa: E402
from test_gpu_kv_many_rows import compare  # noqa: E402

pytestmark = pytest.mark.gpu


def microseconds(call, calls=10, groups=7):
    """Least time of a call, of some groups of calls."""
    for _ in range(3):
        call()
    best = []
    for _ in range(groups):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            call()
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b) * 1e3 / calls)
    return min(best)


def filled(blocks, kv, dim, block):
    cache = qw.kv_cache(blocks, kv, dim, block)
    for c in cache[:2]:
        c.random_(-127, 128)
    for c in cache[2:]:
        c.fill_(0.01)
    return cache


def call_of(new, context, heads, kv, dim, block, max_new=None):
    width = -(-max(context) // block)
    cache = filled(len(new) * width, kv, dim, block)
    table = torch.arange(len(new) * width, dtype=torch.int32, device="cuda:0").view(len(new), width)
    q = torch.randn((sum(new), heads, dim), device="cuda:0").to(F16)
    args = (q, *cache, table, ints(context), ints(np.concatenate([[0], np.cumsum(new)])), max_new or max(new))
    return lambda: qw.kv_attention(*args)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv,dim,block", [(32, 2, 128, 64), (16, 4, 64, 16), (7, 1, 128, 32), (40, 1, 64, 128)])
@pytest.mark.parametrize("new", [[1] * 11 + [8], [8] + [1] * 11, [1, 0, 5, 1, 1, 13, 2, 0, 1, 1, 40, 1], [1] * 30 + [60]])
def test_unequal_new_tokens(new, heads, kv, dim, block, dtype):
    rng = np.random.default_rng(heads + len(new) + new[0])
    context = [int(c) for c in rng.integers(40, 1700, len(new))]
    context[0], context[-1], context[4] = 3000, 2900, 0
    compare(rng, new, context, heads, kv, block, dtype, dim=dim, prompt=False)


@pytest.mark.parametrize("requests", [255, 256, 257, 600])
def test_unequal_new_tokens_of_many_requests(requests):
    rng = np.random.default_rng(requests)
    new = [int(n) for n in rng.integers(0, 2, requests)]
    context = [int(c) for c in rng.integers(0, 90, requests)]
    for at in (1, requests // 2, requests - 1):
        new[at], context[at] = 9 + at % 5, 2500 + at % 70
    compare(rng, new, context, 8, 1, 64, F16, dim=64, prompt=False)


def test_one_draft_beside_decodes_takes_no_multiple_of_the_time():
    """One request with eight new tokens among 63 with one each: what the call
    reads grows by nothing, so its time must not double."""
    context = [8000] * 64
    say("64 decodes, and 63 beside a draft of 8")
    alone = microseconds(call_of([1] * 64, context, 32, 2, 128, 64))
    mixed = microseconds(call_of([8] + [1] * 63, context, 32, 2, 128, 64))
    loose = microseconds(call_of([1] * 64, context, 32, 2, 128, 64, max_new=8))
    print("decodes %.1f us, with a draft %.1f us, with a loose bound %.1f us" % (alone, mixed, loose))
    assert mixed < 2 * alone and loose < 2 * alone
