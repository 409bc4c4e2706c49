"""kv_attention at sizes from which the call takes its kernel for many query
rows (the other sizes are in test_gpu_kv.py), calls with more requests than a
workgroup has threads, kv_write and qk_norm_rope with from few to many tokens
a wave, and a whole step in a replayed graph."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402
from test_gpu_kv import BF16, F16, TYPES, dev, host, ints, same, slots_of, unit, within, write_and_compare  # noqa: E402

DIM = 128


def many_rows(tokens, requests, heads, kv, most):
    """The rule of the call, so that these tests fail if it moves away from
    their sizes."""
    cus, group = torch.cuda.get_device_properties(0).multi_processor_count, heads // kv
    blocks = (tokens * group / 256 + requests) * kv
    units = (tokens * group / 32 + requests) * kv
    return most * group > 32 and 2.3 * max(1.0, blocks / cus) <= 6.0 * units / (8 * cus)


def compare(rng, new, context, heads, kv, block, dtype, causal=True, window=0, scale=None, q=None, cache=None, table=None,
            max_context=None, dim=DIM, prompt=True):
    new, context = list(new), list(context)
    say("attention T=%d R=%d new=%s ctx=%s %d/%d D=%d B=%d %s causal=%s window=%d" % (
        sum(new), len(new), new[:9], context[:9], heads, kv, dim, block, dtype, causal, window))
    assert not prompt or many_rows(sum(new), len(new), heads, kv, max(new))
    made, blocks = ref.pages(rng, context, block)
    table = made if table is None else table
    cache = ref.random_cache(rng, blocks, kv, dim, block) if cache is None else cache
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    q = dev(rng.standard_normal((T, heads, dim)) * 1.5, dtype) if q is None else q
    out = torch.full((T, heads, dim), float("nan"), dtype=dtype, device="cuda:0")
    got = qw.kv_attention(q, *[dev(c) for c in cache], ints(table), ints(context), ints(cu), max(new), max_context=max_context,
                          scale=scale, causal=causal, window=window, out=out)
    real = dim ** -0.5 if scale is None else scale
    bound = context if max_context is None else np.minimum(context, max_context)
    want, mass, reach, tail = ref.attention_rows(host(q), cache, table, bound, cu, max(new), real, causal, window)
    within(host(got), want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(dtype)))
    return got


RAGGED = [1, 70, 0, 33, 129, 64, 2, 101]


def test_rows_reference_is_the_reference():
    rng = np.random.default_rng(3)
    for causal, window in ((True, 0), (True, 20), (False, 7), (False, 0)):
        new, context = [9, 1, 4, 3, 0], [3, 0, 40, 90, 5]
        table, blocks = ref.pages(rng, context, 16)
        table[2, 1], table[3, 0], table[3, 3] = -1, blocks, 2 ** 31 - 1
        cache = ref.random_cache(rng, blocks, 2, 64, 16)
        q, cu = rng.standard_normal((17, 6, 64)), np.concatenate([[0], np.cumsum(new)])
        for most in (9, 3):
            a = ref.attention(q, cache, table, context, cu, most, 0.2, causal, window)
            b = ref.attention_rows(q, cache, table, context, cu, most, 0.2, causal, window)
            for x, y in zip(a, b):
                np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_prompts(block, dtype):
    compare(np.random.default_rng(block), RAGGED, RAGGED, 64, 8, block, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,new", [(64, 64, [300, 37, 129]), (40, 8, [90, 64, 255, 1, 200]), (64, 2, [1, 51, 52, 100, 300]),
                                          (48, 16, [250, 31, 222, 5]), (28, 4, [1000, 33])])
def test_groups(heads, kv, new):
    rng = np.random.default_rng(heads)
    compare(rng, new, [n + p for n, p in zip(new, (0, 65, 700, 3, 200))], heads, kv, 32, F16)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 15, 64, 333])
@pytest.mark.parametrize("block", [16, 128])
def test_chunks_and_windows(block, window, causal):
    context = [1, 300, 0, 33, 700, 640, 1000, 102]
    compare(np.random.default_rng(block + window), RAGGED, context, 64, 8, block, BF16, causal=causal, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 4500])
@pytest.mark.parametrize("ctx", [2048, 2049, 4095, 4096, 4097, 6208, 12500])
def test_long_contexts(ctx, window):
    """Around whole and half segments of scales (64 tiles of 64 keys)."""
    compare(np.random.default_rng(ctx), [40, 300, 100], [ctx, 300, 164], 64, 8, 64, F16, window=window)


@pytest.mark.gpu
def test_rows_that_see_nothing():
    rng = np.random.default_rng(1)
    new, context = [90, 1, 70, 200, 60], [30, 0, 140, 220, 0]
    table, blocks = ref.pages(rng, context, 16)
    table[2, :] = -1
    got = host(compare(rng, new, context, 64, 8, 16, F16, table=table, cache=ref.random_cache(rng, blocks, 8, DIM, 16)))
    assert not got[:60].any() and got[60:90].any() and not got[90:161].any() and not got[361:].any()


@pytest.mark.gpu
def test_missing_blocks_in_the_middle():
    rng = np.random.default_rng(2)
    context = [400, 190, 300]
    table, blocks = ref.pages(rng, context, 16)
    table[0, 3], table[0, 7], table[1, 0], table[0, 24], table[2, 4:8] = -1, blocks, 2 ** 31 - 1, -5, -1
    compare(rng, [300, 2, 150], context, 64, 8, 16, F16, table=table, cache=ref.random_cache(rng, blocks, 8, DIM, 16))


@pytest.mark.gpu
def test_scales_far_apart():
    rng = np.random.default_rng(40)
    context = [400, 350]
    table, blocks = ref.pages(rng, context, 16)
    k, v, ks, vs = ref.random_cache(rng, blocks, 8, DIM, 16)
    ks *= np.float32(2.0 ** -4)
    vs *= (2.0 ** rng.uniform(-20, 0, vs.shape)).astype(np.float32)
    dead = table[0, [2, 5, 6]]
    vs[dead], v[dead] = 0, 0
    ks[table[0, 9]], k[table[0, 9]] = 0, 0
    compare(rng, [200, 300], context, 64, 8, 16, BF16, cache=(k, v, ks, vs), table=table)
    vs[:], v[:] = 0, 0
    assert not host(compare(rng, [200, 300], context, 64, 8, 16, F16, cache=(k, v, ks, vs), table=table)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_peaked_and_flat(dtype):
    """Scores in the hundreds (one key takes all, the reference moves often),
    scores of zero, and one large weight beside many tiny ones."""
    rng = np.random.default_rng(7)
    for gain in (40.0, 4.0, 0.0):
        q = dev(rng.standard_normal((450, 64, DIM)) * gain, dtype)
        compare(rng, [250, 200], [333, 200], 64, 8, 64, dtype, q=q)


@pytest.mark.gpu
def test_bf16_range():
    rng = np.random.default_rng(11)
    for power in (-60, 60):
        q = dev(rng.standard_normal((450, 64, DIM)) * 2.0 ** power, BF16)
        table, blocks = ref.pages(rng, [500], 32)
        k, v, ks, vs = ref.random_cache(rng, blocks, 8, DIM, 32)
        compare(rng, [450], [500], 64, 8, 32, BF16, q=q, table=table, cache=(k, v, (ks * 2.0 ** -power).astype(np.float32), vs))


@pytest.mark.gpu
@pytest.mark.parametrize("block", [16, 64])
def test_hidden_garbage(block):
    """NaN and infinite scales in other requests' blocks; -128 codes behind
    the context's end, also where the tile goes on for blocks."""
    rng = np.random.default_rng(13)
    context = [70, 129, 300]
    table, blocks = ref.pages(rng, context, block, spare=4)
    k, v, ks, vs = ref.random_cache(rng, blocks, 8, DIM, block)
    used = set(table[table >= 0].tolist())
    for b in range(blocks):
        if b not in used:
            ks[b], vs[b] = np.nan, np.inf
    last = table[0, 69 // block]
    k[last, :, 69 % block + 1:], v[last, :, :, 69 % block + 1:] = -128, -128
    # what was in LDS before must not matter either: a call full of NaN queries goes first
    bad = dev(np.full((430, 64, DIM), np.nan), F16)
    on = [dev(c) for c in (k, v, ks, vs)]
    qw.kv_attention(bad, *on, ints(table), ints(context), ints([0, 70, 170, 430]), 260)
    compare(rng, [70, 100, 260], context, 64, 8, block, F16, cache=(k, v, ks, vs), table=table)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv", [(64, 8), (64, 64)])
def test_nan_and_inf_queries_stay_in_their_row(heads, kv):
    rng = np.random.default_rng(17)
    q = rng.standard_normal((450, heads, DIM))
    clean = dev(q, F16)
    q[0, 1, 5], q[100, 9, 7], q[-1, 0, 0] = np.nan, np.nan, np.inf
    dirty = dev(q, F16)
    context, cu = [450, 90], [0, 400, 450]
    assert many_rows(450, 2, heads, kv, 400)
    table, blocks = ref.pages(rng, context, 32)
    cache = [dev(c) for c in ref.random_cache(rng, blocks, kv, DIM, 32)]
    say("attention with NaN queries %d/%d" % (heads, kv))
    a, b = (host(qw.kv_attention(x, *cache, ints(table), ints(context), ints(cu), 400)) for x in (clean, dirty))
    keep = np.ones(b.shape[:2], bool)
    for at in ((0, 1), (100, 9), (-1, 0)):
        assert np.isnan(b[at]).all()
        keep[at] = False
    assert np.array_equal(a[keep], b[keep])


@pytest.mark.gpu
def test_scale_signs_and_zero():
    for scale in (0.0, -0.1, 0.3):
        compare(np.random.default_rng(19), [300, 120], [320, 300], 64, 8, 32, F16, scale=scale)


@pytest.mark.gpu
def test_strided_queries_bounds_and_other_rows():
    rng = np.random.default_rng(23)
    T, heads, kv, block = 440, 64, 8, 16
    fused = dev(rng.standard_normal((T, (heads + 2 * kv) * DIM)), F16)
    q = fused[:, :heads * DIM].view(T, heads, DIM)
    compare(rng, [400, 40], [400, 90], heads, kv, block, F16, q=q)
    compare(rng, [400, 40], [433, 90], heads, kv, block, F16, q=q, max_context=77)
    # rows of no request keep what they hold, and offsets that are none stay inside the tensors
    table, blocks = ref.pages(rng, [440], block)
    cache = [dev(c) for c in ref.random_cache(rng, blocks, kv, DIM, block)]
    out = torch.full((T, heads, DIM), 7.0, dtype=F16, device="cuda:0")
    say("attention rows of no request")
    qw.kv_attention(q, *cache, ints(table), ints([440]), ints([5, 435]), 420, out=out)
    got = host(out)
    assert (got[:5] == 7).all() and (got[425:] == 7).all() and not (got[5:425] == 7).all(-1).any()
    say("attention, offsets outside")
    qw.kv_attention(q, *cache, ints(table), ints([10 ** 9]), ints([-5, 10 ** 9]), 440, out=out)
    qw.kv_attention(q, *cache, ints(table), ints([-40]), ints([8, 2]), 440, out=out)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [511, 512, 513, 1100])
def test_prompts_of_many_requests(requests):
    """More requests than a workgroup has threads, most with one token or none."""
    rng = np.random.default_rng(requests)
    new = [int(n) for n in rng.integers(0, 2, requests)]
    for at in (0, 3, requests // 2, requests - 1):
        new[at] = 1000 + at % 50
    compare(rng, new, [n + int(p) for n, p in zip(new, rng.integers(0, 30, requests))], 64, 2, 64, F16)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 1), (64, 5)])
@pytest.mark.parametrize("requests", [255, 256, 257, 600])
def test_decode_of_many_requests(requests, dim, new):
    """More requests than a batch of the scan that deals out ranges of keys."""
    rng = np.random.default_rng(requests + dim)
    context = [int(c) for c in rng.integers(0, 90, requests)]
    for at in (1, requests // 2, requests - 1):
        context[at] = 2500 + at % 70
    compare(rng, [new] * requests, context, 16, 2, 64, F16, dim=dim, prompt=False)


@pytest.mark.gpu
def test_same_bits_and_streams():
    rng = np.random.default_rng(31)
    new, context = [300, 150], [1000, 150]
    table, blocks = ref.pages(rng, context, 64)
    on = [dev(c) for c in ref.random_cache(rng, blocks, 8, DIM, 64)]
    q = dev(rng.standard_normal((450, 64, DIM)), F16)
    args = (q, *on, ints(table), ints(context), ints([0, 300, 450]), 300)
    assert many_rows(450, 2, 64, 8, 300)
    say("attention of many rows twice, and on another stream")
    first = qw.kv_attention(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = qw.kv_attention(*args)
    third = qw.kv_attention(*args)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)
    # a row's result does not depend on the rows beside it
    alone = qw.kv_attention(q[300:], *on, ints(table[1:]), ints(context[1:]), ints([0, 150]), 150)
    if many_rows(150, 1, 64, 8, 150):
        assert torch.equal(first[300:], alone)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,dim", [(511, 128), (512, 64), (513, 128), (2500, 64), (4096, 128), (4097, 64), (6000, 128)])
def test_write_windows(tokens, dim, block, dtype):
    """Windows of 4, 16 and 64 tokens over single tokens, short runs and long
    ones, beginning and ending anywhere, with padding between requests."""
    rng = np.random.default_rng(tokens + block)
    fresh = []
    while sum(fresh) < tokens:
        n = int(rng.choice([1, 1, 1, 2, 7, 15, 16, 17, 40, 64, 130, 300]))
        fresh.append(min(n, tokens - sum(fresh)))
    past = [int(x) for x in rng.integers(0, 2 * block, len(fresh))]
    context = [p + n for p, n in zip(past, fresh)]
    table, blocks = ref.pages(rng, context, block)
    slots = []
    for r in range(len(fresh)):
        slots += slots_of(table, r, past[r], context[r], block)
    cut = int(np.cumsum(fresh)[len(fresh) // 2])
    for at in (tokens, cut, 0):   # padding takes the place of tokens at the end
        slots[at:at] = [-1, blocks * block, -7][:1 + at % 3]
    write_and_compare(rng, slots, 2, dim, block, blocks, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,pairs,norm", [
    (1, 70, 9, 64, 64, False, True), (2, 33, 1, 128, 128, True, True), (700, 5, 3, 128, 64, False, False),
    (3000, 9, 2, 64, 64, False, True), (8192, 4, 1, 128, 96, True, True), (8300, 7, 2, 64, 32, False, True)])
def test_norm_rope_waves(tokens, hq, hk, dim, rot, pairs, norm, dtype):
    """From many waves a token to one for all of its heads; infinities in the
    channels that do not turn, and in a row beside, stay where they are."""
    rng = np.random.default_rng(tokens + dim + rot)
    span = 64
    say("norm_rope T=%d %d/%d D=%d rot=%d pairs=%s norm=%s %s" % (tokens, hq, hk, dim, rot, pairs, norm, dtype))
    q, k = (dev(rng.standard_normal((tokens, h, dim)), dtype) for h in (hq, hk))
    pos = rng.integers(-2, span + 1, tokens)
    pos[0] = 5
    angle = rng.uniform(0, 7, (span, rot // 2))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    wq, wk = (dev(1 + 0.3 * rng.standard_normal(dim), dtype) for _ in range(2)) if norm else (None, None)
    args = (ints(pos), dev(cos), dev(sin), wq, wk)
    got = qw.qk_norm_rope(q, k, *args, eps=1e-5, interleaved=pairs)
    for g, x, w in zip(got, (q, k), (wq, wk)):
        want, mag = ref.norm_rope(host(x), pos, cos, sin, None if w is None else host(w), 1e-5, pairs)
        within(host(g), want, unit(dtype) * np.abs(want) + (dim + 8) * 2.0 ** -24 * mag + 2.0 ** -25)
    bad = q.clone()
    bad[0, 1, dim - 1] = float("inf")
    other = qw.qk_norm_rope(bad, k, *args, eps=1e-5, interleaved=pairs)
    a, b = host(got[0]), host(other[0])
    same(b[0, 2:], a[0, 2:], "the heads beside")
    same(b[1:], a[1:], "the tokens beside")
    same(host(other[1]), host(got[1]), "the keys")
    if not norm and rot < dim:
        same(b[0, 1, :dim - 1], a[0, 1, :dim - 1], "the other channels")
        assert np.isinf(b[0, 1, dim - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("new,heads,kv,dim", [(1, 16, 2, 64), (4, 16, 4, 128), (150, 64, 8, 128)])
def test_step_in_a_replayed_graph(new, heads, kv, dim):
    """Plan, rotation, write and attention captured once and replayed over
    growing requests, with eager work between, against the eager calls."""
    rng = np.random.default_rng(new)
    R, block, steps = 3, 32, 4
    width = (700 + steps * new) // block + 2
    past0 = [0, 40, 690]
    T = R * new
    assert new < 100 or many_rows(T, R, heads, kv, new)

    def fresh_state():
        free = ints(np.random.default_rng(5).permutation(R * width))
        table = torch.full((R, width), -1, dtype=torch.int32, device="cuda:0")
        cache = qw.kv_cache(R * width, kv, dim, block)
        begin = qw.kv_plan(ints([0] * R), ints(past0), table, free, block, sum(past0))
        k, v = (dev(np.random.default_rng(6 + i).standard_normal((sum(past0), kv, dim)), F16) for i in range(2))
        qw.kv_write(k, v, begin.slots, *cache)
        return table, free[int(begin.counts[0].item()):].contiguous(), cache

    def step(past, table, free, cache, x, tables):
        plan = qw.kv_plan(past, fresh, table, free, block, T)
        q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        q, k = qw.qk_norm_rope(q, k, plan.positions, *tables)
        qw.kv_write(k, v, plan.slots, *cache)
        o = qw.kv_attention(q, *cache, plan.block_table, plan.context, plan.cu_tokens, new, max_context=width * block)
        return plan, o

    fresh = ints([new] * R)
    angle = np.arange(1000)[:, None] * 0.01 ** (np.arange(dim // 2) / (dim // 2))
    tables = (dev(np.cos(angle).astype(np.float32)), dev(np.sin(angle).astype(np.float32)))
    xs = [dev(rng.standard_normal((T, heads + 2 * kv, dim)), F16) for _ in range(steps)]
    say("eager steps of %d x %d tokens" % (R, new))
    table, free, cache = fresh_state()
    eager, taken, past = [], 0, np.array(past0)
    for x in xs:
        plan, o = step(ints(past), table, free[taken:].contiguous(), cache, x, tables)
        eager.append(host(o))
        taken += int(plan.counts[0].item())
        past = past + new
    eager_cache = [host(c) for c in cache]

    say("the same steps from a graph")
    table, free, cache = fresh_state()
    state = (ints(past0), torch.full((R * width,), -1, dtype=torch.int32, device="cuda:0"), xs[0].clone())
    scratch = (torch.full_like(table, -1), state[1], qw.kv_cache(R * width, kv, dim, block))
    step(ints([0] * R), scratch[0], free, scratch[2], state[2], tables)   # (loads every kernel)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, o = step(state[0], table, state[1], cache, state[2], tables)
    taken, past = 0, np.array(past0)
    for i, x in enumerate(xs):
        state[0].copy_(ints(past))
        state[1].fill_(-1)
        left = free[taken:]
        state[1][:left.shape[0]].copy_(left)
        state[2].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(o), eager[i]), "replay %d" % i
        taken += int(plan.counts[0].item())
        past = past + new
        (x.float() * 2).sum().item()
    for a, b in zip(cache, eager_cache):
        assert np.array_equal(host(a), b)
