"""The softmax weights of kv_attention where one key takes most of the mass:
the many small ones behind it still make the output, and must keep their bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import TYPES, dev, host, ints, unit, within  # noqa: E402
from test_gpu_kv_many_rows import compare, many_rows  # noqa: E402

pytestmark = pytest.mark.gpu


def sink(new, ctx, heads, kv, dim, block, dtype, many):
    """Key 0 of each head scores `gap` (another one for each query head) and has
    value codes 0; all other keys score 0 exactly, with codes of 64 to 127."""
    rng = np.random.default_rng(ctx + dim)
    assert many == (dim == 128 and many_rows(new, 1, heads, kv, new))
    table, blocks = ref.pages(rng, [ctx], block)
    k = np.zeros((blocks, kv, block, dim), np.int8)
    v = rng.integers(64, 128, (blocks, kv, dim, block)).astype(np.int8)
    ks, vs = np.full((blocks, kv), 2.0 ** -4, np.float32), np.full((blocks, kv), 2.0 ** -6, np.float32)
    k[table[0, 0], :, 0, 0], v[table[0, 0], :, :, 0] = 127, 0
    # gaps from 14 to 26 powers of two, at no regular distance
    gap = np.log(2.0) * (14 + 12 * ((np.arange(heads) * 0.6180339887 + 0.21) % 1.0))
    scale = dim ** -0.5
    q = np.zeros((new, heads, dim))
    q[:, :, 0] = gap / (scale * 127 * 2.0 ** -4)
    q = dev(q, dtype)
    say("attention behind a dominant key: new=%d ctx=%d %d/%d D=%d %s" % (new, ctx, heads, kv, dim, dtype))
    got = host(qw.kv_attention(q, dev(k), dev(v), dev(ks), dev(vs), ints(table), ints([ctx]), ints([0, new]), new))
    real = host(q)[0, :, 0] * scale * 127 * 2.0 ** -4                     # the gaps as rounded to the type
    codes = v[table[0].astype(np.int64)].astype(np.float64).transpose(1, 2, 0, 3).reshape(kv, dim, -1)[:, :, :ctx] * 2.0 ** -6
    upto = np.cumsum(codes, 2)[:, :, ctx - new:].transpose(2, 0, 1).repeat(heads // kv, 1)   # [new, heads, dim]
    keys = np.arange(ctx - new, ctx)[:, None, None]                       # behind the first one
    want = upto / (np.exp(real)[None, :, None] + keys)
    # each weight to fp16, with the largest at 2^8 or more: 2^-11 of it, or 2^-25 of what lies 8 powers above the sink's
    small = np.exp(-real)[None, :, None]
    step = np.maximum(2.0 ** -11, 2.0 ** -33 / small)
    # the scores' products and sums in fp32, as a relative error of the weights; then the output's rounding
    tol = want * (step * (1 + 2.0 ** -8) + 2 * (dim + 8) * 2.0 ** -24 * real[None, :, None] + unit(dtype) * (1 + 2.0 ** -8)) + 2.0 ** -25
    within(got, want, tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,heads,kv,dim,block", [(1, 8, 2, 64, 16), (1, 32, 2, 128, 64), (5, 32, 8, 128, 32), (40, 16, 16, 64, 128)])
def test_dominant_first_key(new, heads, kv, dim, block, dtype):
    sink(new, 16384 + new, heads, kv, dim, block, dtype, False)


@pytest.mark.parametrize("dtype", TYPES)
def test_dominant_first_key_many_rows(dtype):
    sink(450, 16384 + 450, 64, 8, 128, 64, dtype, True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,heads,kv,dim,prompt", [(1, 4, 2, 64, False), (40, 4, 2, 128, False), (450, 64, 8, 128, True)])
def test_value_scales_over_forty_powers(new, heads, kv, dim, prompt, dtype):
    """Blocks whose value scales lie up to 2^40 apart, and one of zeros."""
    rng = np.random.default_rng(new)
    context = [new + 700]
    table, blocks = ref.pages(rng, context, 16)
    k, v, ks, vs = ref.random_cache(rng, blocks, kv, dim, 16)
    vs *= (2.0 ** rng.uniform(-40, 0, vs.shape)).astype(np.float32)
    vs[table[0, 5]], v[table[0, 5]] = 0, 0
    compare(rng, [new], context, heads, kv, 16, dtype, dim=dim, table=table, cache=(k, v, ks, vs), prompt=prompt)
