"""Outputs that the calls allocate are contiguous whatever the strides of
their inputs, and hold the same bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
from test_gpu_kv import BF16, F16, dev, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,hq,hk,dim", [(1, 4, 2, 64), (1, 1, 1, 128), (3, 6, 1, 64), (5, 8, 2, 128)])
def test_outputs_of_views(tokens, hq, hk, dim, dtype):
    rng = np.random.default_rng(tokens + hq)
    fused = dev(rng.standard_normal((tokens, hq + 2 * hk + 3, dim)), dtype)
    q, k, v = fused[:, 1:1 + hq], fused[:, 1 + hq:1 + hq + hk], fused[:, 2 + hq + hk:2 + hq + 2 * hk]
    cos = torch.rand((9, dim // 2), device="cuda:0")
    pos = ints(np.arange(tokens))
    views = qw.qk_norm_rope(q, k, pos, cos, cos)
    plain = qw.qk_norm_rope(q.contiguous(), k.contiguous(), pos, cos, cos)
    for a, b in zip(views, plain):
        assert a.is_contiguous() and a.shape == b.shape and torch.equal(a, b)
    cache = qw.kv_cache(2, hk, dim, 16)
    qw.kv_write(k, v, ints(16 + np.arange(tokens)), *cache)
    args = (*cache, ints([[1]]), ints([tokens]), ints([0, tokens]), tokens)
    a, b = qw.kv_attention(q, *args), qw.kv_attention(q.contiguous(), *args)
    assert a.is_contiguous() and a.shape == (tokens, hq, dim) and torch.equal(a, b)
    assert a.view(tokens, -1).data_ptr() == a.data_ptr()
