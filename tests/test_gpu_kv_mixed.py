"""kv_attention over requests whose numbers of new tokens differ: results, and
that one request with more of them does not make the others slow."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
from gpu_util import say  # noqa: E402
import kv_reference as ref  # noqa: E402
from test_gpu_kv import BF16, F16, TYPES, dev, ints  # noqa: E402
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
    blocks = min(len(new) * width, (2 ** 32 if dim == 128 else 2 ** 31) // (kv * dim * block))   # (shared, if there are too many)
    cache = filled(blocks, kv, dim, block)
    table = (torch.arange(len(new) * width, dtype=torch.int32, device="cuda:0") % blocks).view(len(new), width)
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


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 4000), (False, 4000), (True, 50)])
@pytest.mark.parametrize("dtype", TYPES)
def test_prompts_beside_tokens_behind_long_contexts(dtype, causal, window):
    """Requests with few rows and with many in one call: up to 128 new tokens of 8
    heads a key head go one way, more of them the other."""
    rng = np.random.default_rng(window)
    new, past = [450, 1, 128, 0, 129, 1, 4, 33, 1], [0, 5000, 4100, 77, 30, 0, 6000, 4500, 2]
    compare(rng, new, [n + p for n, p in zip(new, past)], 64, 8, 32, dtype, causal=causal, window=window)


@pytest.mark.parametrize("heads,kv,dim,tokens", [(16, 16, 64, 2100), (40, 1, 64, 1800), (64, 1, 128, 300), (48, 16, 128, 700)])
def test_groups_of_heads_beside_long_contexts(heads, kv, dim, tokens):
    rng = np.random.default_rng(heads)
    few = max(1, 1024 // (heads // kv))
    new = [tokens, 1, few, few + 1, 0, 1]
    past = [5, tokens + 3000, tokens + 2500, tokens + 2600, 9, 40]
    compare(rng, new, [n + p for n, p in zip(new, past)], heads, kv, 16, BF16, dim=dim, prompt=False)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 70)])
@pytest.mark.parametrize("requests,heads,kv,dim,most", [(41, 16, 16, 64, 200), (300, 16, 16, 64, 130), (256, 12, 2, 64, 400),
                                                        (60, 32, 2, 128, 33)])
def test_few_of_the_row_blocks_are_there(requests, heads, kv, dim, most, causal, window):
    """Requests with one or no new token, and two with many: the row blocks of
    all of them in a row, more requests than a workgroup has threads among them."""
    rng = np.random.default_rng(requests)
    new = [int(n) for n in rng.integers(0, 2, requests)]
    new[1], new[requests - 1] = most - 1, most
    context = [n + int(p) for n, p in zip(new, rng.integers(0, 90, requests))]
    compare(rng, new, context, heads, kv, 64, F16, causal=causal, window=window, dim=dim, prompt=False)


@pytest.mark.parametrize("requests,heads,kv,dim", [(200, 16, 16, 64), (1100, 4, 2, 128)])
def test_many_tokens_and_one_long_context(requests, heads, kv, dim):
    rng = np.random.default_rng(requests)
    context = [int(c) for c in rng.integers(0, 60, requests)]
    context[7], context[requests // 2] = 9000, 4500
    compare(rng, [1] * requests, context, heads, kv, 64, F16, dim=dim, prompt=False)


@pytest.mark.parametrize("what,heads,kv,dim,first,second", [
    ("a prompt beside one token", 32, 2, 128, ([4096], [4096]), ([1], [131072])),
    ("a prompt beside a draft", 32, 2, 128, ([4096], [4096]), ([8], [131072])),
    ("a prompt beside 63 tokens", 32, 2, 128, ([512], [512]), ([1] * 63, [8000] * 63)),
    ("a prompt beside one token, 64 channels", 16, 16, 64, ([4096], [4096]), ([1], [131072])),
    ("a prompt beside 255 tokens, 64 channels", 16, 16, 64, ([4096], [4096]), ([1] * 255, [500] * 255)),
    ("192 tokens, one far behind", 16, 16, 64, ([1] * 191, [1000] * 191), ([1], [131072])),
])
def test_a_long_context_is_shared_out(what, heads, kv, dim, first, second):
    """One call for both kinds of requests takes no multiple of two calls' time."""
    say(what)
    one, two = (microseconds(call_of(*x, heads, kv, dim, 64)) for x in (first, second))
    both = microseconds(call_of(first[0] + second[0], first[1] + second[1], heads, kv, dim, 64))
    print("%s: %.1f and %.1f us alone, %.1f us together" % (what, one, two, both))
    assert both < 1.7 * (one + two)


@pytest.mark.parametrize("new,past,heads,kv,dim", [
    ([450, 1, 3, 200], [0, 5000, 4100, 30], 64, 8, 128),              # many rows, and few in ranges
    ([2100, 1, 1024, 3], [5, 5100, 30, 4000], 16, 16, 64),            # a workgroup a unit, and few in ranges
    ([199, 200] + [1] * 39, [10] * 41, 16, 16, 64),                   # the row blocks in a row
    ([1] * 30 + [60], [1500] * 31, 32, 2, 128),                       # joined by ranges
])
def test_a_captured_call(new, past, heads, kv, dim):
    """One graph, replayed over other queries and contexts with eager work
    between, against the eager calls."""
    rng = np.random.default_rng(len(new))
    top = np.array(new) + np.array(past)
    table, blocks = ref.pages(rng, [int(c) for c in top], 32)
    on = [dev(c) for c in ref.random_cache(rng, blocks, kv, dim, 32)]
    q = torch.zeros((sum(new) + 3, heads, dim), dtype=F16, device="cuda:0")
    context, tab, cu = ints(top), ints(table), ints(np.concatenate([[0], np.cumsum(new)]))
    steps = [(dev(rng.standard_normal(q.shape), F16), ints(np.maximum(new, top - rng.integers(0, 40, len(new))))) for _ in range(3)]
    call = lambda: qw.kv_attention(q, *on, tab, context, cu, max(new), max_context=int(top.max()))  # noqa: E731
    eager = []
    for x, c in steps:
        q.copy_(x)
        context.copy_(c)
        eager.append(call())
    torch.cuda.synchronize()
    say("a captured call of %d requests, D=%d" % (len(new), dim))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for again in range(2):
        for (x, c), want in zip(steps, eager):
            q.copy_(x)
            context.copy_(c)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and not out[-3:].any()
            (x.float() * 2).sum().item()
