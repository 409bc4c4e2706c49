"""Where two calls take the same kernel and give a row's keys to one workgroup,
the row's bits do not depend on the requests beside it."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import TYPES, dev, ints  # noqa: E402
from test_gpu_kv_many_rows import many_rows  # noqa: E402

pytestmark = pytest.mark.gpu


def alone_and_beside(new, context, at, heads, kv, dim, dtype):
    rng = np.random.default_rng(sum(new))
    table, blocks = ref.pages(rng, context, 64)
    on = [dev(c) for c in ref.random_cache(rng, blocks, kv, dim, 64)]
    cu = np.concatenate([[0], np.cumsum(new)])
    q = dev(rng.standard_normal((sum(new), heads, dim)) * 1.5, dtype)
    say("attention of request %d of new=%s alone and beside the others, D=%d" % (at, new, dim))
    # (max_context: neither call may take ranges)
    beside = qw.kv_attention(q, *on, ints(table), ints(context), ints(cu), max(new), max_context=max(context))
    rows = slice(int(cu[at]), int(cu[at + 1]))
    alone = qw.kv_attention(q[rows], *on, ints(table[at:at + 1]), ints(context[at:at + 1]), ints([0, new[at]]), new[at],
                            max_context=context[at])
    assert torch.equal(beside[rows], alone)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows(dtype):
    new, context = [300, 600], [1000, 900]
    assert many_rows(900, 2, 64, 8, 600) and many_rows(600, 1, 64, 8, 600)
    alone_and_beside(new, context, 1, 64, 8, 128, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,context,at", [([100, 30, 200, 1], [500, 30, 200, 400], 0), ([40, 200], [500, 200], 1),
                                            ([90] + [1] * 40, [300] + [30] * 40, 0)])
def test_one_workgroup_a_unit(new, context, at, dtype):
    alone_and_beside(new, context, at, 8, 2, 64, dtype)
