"""Rows of kv_attention's output that belong to no request: zero where the call
allocates the output, kept where the caller gives one."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import F16, dev, ints  # noqa: E402

pytestmark = pytest.mark.gpu

# (heads, key heads, channels, tokens, offsets, contexts, max_new)
CASES = {
    "one workgroup a unit": (4, 2, 64, 9, [2, 5, 6], [40, 60], 3),
    "ranges": (8, 2, 64, 6, [1, 2, 3], [3000, 1700], 1),
    "many rows": (64, 8, 128, 1000, [5, 455, 655], [455, 300], 450),
    "many rows, and few": (64, 8, 128, 1000, [300, 301, 900], [6000, 700], 599),
    "many rows, requests without tokens": (64, 8, 128, 1000, [0, 0, 450], [3, 450], 450),
    "ranges, a batch of requests": (4, 2, 64, 261, list(range(2, 259)), [3000, 20] * 128, 1),
    "ranges, more than a batch": (4, 2, 64, 270, list(range(2, 260)), [20, 3000, 0] * 85 + [7, 9], 1),
    "few of the row blocks": (16, 16, 64, 300, [5] + list(range(205, 246)), [300] + [30] * 40, 200),
    "no request has tokens": (4, 2, 64, 7, [0, 0, 0], [40, 60], 3),
}


def args_of(case):
    heads, kv, dim, tokens, cu, context, max_new = CASES[case]
    rng = np.random.default_rng(tokens)
    table, blocks = ref.pages(rng, context, 32)
    cache = [dev(c) for c in ref.random_cache(rng, blocks, kv, dim, 32)]
    q = dev(rng.standard_normal((tokens, heads, dim)), F16)
    computed = np.zeros(tokens, bool)
    for a, b in zip(cu, cu[1:]):
        computed[a:b] = True
    return (q, *cache, ints(table), ints(context), ints(cu), max_new), computed


@pytest.mark.parametrize("case", CASES)
def test_rows_of_no_request(case):
    args, computed = args_of(case)
    say("attention with rows of no request: " + case)
    kept = qw.kv_attention(*args, out=torch.full_like(args[0], 7.0))
    torch.cuda.synchronize()
    hole = torch.full_like(args[0], float("nan"))   # the allocation that the next output takes
    at = hole.data_ptr()
    del hole
    made = qw.kv_attention(*args)
    torch.cuda.synchronize()
    assert made.data_ptr() == at
    rest = torch.from_numpy(~computed).cuda()
    assert (kept[rest] == 7).all() and (made[rest] == 0).all()
    assert torch.equal(made[~rest], kept[~rest])


@pytest.mark.parametrize("requests,max_new", [(0, 3), (2, 0)])
def test_nothing_to_compute(requests, max_new):
    args, _ = args_of("one workgroup a unit")
    q, kc, vc, ks, vs, table, context, cu, _ = args
    hole = torch.full_like(q, float("nan"))
    del hole
    out = qw.kv_attention(q, kc, vc, ks, vs, table[:requests], context[:requests], cu[:requests + 1], max_new)
    assert out.shape == q.shape and (out == 0).all()
