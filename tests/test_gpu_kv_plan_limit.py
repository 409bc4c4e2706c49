"""kv_plan with as many requests as it takes."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from test_gpu_kv import run_plan  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests", [4096, 8190, qw.KV_PLAN_MAX_REQUESTS])
def test_plan_of_most_requests(requests):
    rng = np.random.default_rng(requests)
    block = 16
    past = rng.integers(0, 3 * block, requests)
    past[-4:] = [block, block - 1, 0, 2 * block + 3]      # in the last batch of the sums: an edge, before it, none, inside
    fresh = rng.integers(0, 4, requests)
    fresh[-4:] = [1, 2, 3 * block, 0]
    table, _ = ref.pages(rng, past, block)
    table = np.concatenate([table, np.full((requests, 4), -1, np.int32)], 1)
    need = int(sum(-(-(p + n) // block) - -(-p // block) for p, n in zip(past, fresh)))
    free = 50000 + rng.permutation(need + 3)
    total = int(fresh.sum())
    run_plan(past, fresh, table, free, block, total)
    run_plan(past, fresh, table, free, block, total + 1030)
    run_plan(past, fresh, table, free[:need // 2], block, total - 5)
