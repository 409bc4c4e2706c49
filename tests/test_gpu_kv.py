"""The paged int8 KV cache operators on the GPU against plain 64-bit
implementations (kv_reference.py)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402
import kv_reference as ref  # noqa: E402
from gpu_util import say  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TYPES = [F16, BF16]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dtype is None else t.to(dtype)


def ints(a):
    return dev(np.asarray(a, dtype=np.int32))


def host(t):
    torch.cuda.synchronize()
    t = t.cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def unit(dtype):
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# kv_plan
# ---------------------------------------------------------------------------

def same(got, want, what):
    bad = np.argwhere(got != want) if got.shape == want.shape else [got.shape]
    assert len(bad) == 0, "%s: %d differ, first at %s" % (what, len(bad), bad[0])


def within(got, want, tol, what=""):
    over = np.abs(got - want) > tol   # NaN is over nothing: looked for apart
    assert not np.isnan(got).any() and not over.any(), "%s: %d NaN, %d out of bound, worst %.3g of it" % (
        what, np.isnan(got).sum(), over.sum(), np.nanmax(np.abs(got - want) / tol))


def run_plan(past, fresh, table, free, block, max_tokens):
    say("plan R=%d B=%d max_tokens=%d" % (len(past), block, max_tokens))
    want = ref.plan(past, fresh, table, free, block, max_tokens)
    got = qw.kv_plan(ints(past), ints(fresh), ints(table), ints(free), block, max_tokens)
    for name, g in zip(("table", "cu", "context", "positions", "slots", "counts"), got):
        same(host(g), want[name], name)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("requests", [1, 7, 255, 256, 257, 700])
def test_plan(requests, block):
    rng = np.random.default_rng(requests * 1000 + block)
    past = rng.integers(0, 3 * block, requests)
    past[rng.random(requests) < 0.2] = 0
    past[rng.random(requests) < 0.2] = block          # an edge
    fresh = rng.integers(0, 2 * block + 2, requests)
    fresh[rng.random(requests) < 0.3] = 0
    fresh[rng.random(requests) < 0.3] = 1
    table, blocks = ref.pages(rng, past, block)
    table = np.concatenate([table, np.full((requests, 4), -1, np.int32)], 1)
    need = int(sum(-(-(p + n) // block) - -(-p // block) for p, n in zip(past, fresh)))
    free = 10000 + rng.permutation(need + 3)
    total = int(fresh.sum())
    run_plan(past, fresh, table, free, block, total)              # exact
    run_plan(past, fresh, table, free, block, total + 1030)       # padding
    run_plan(past, fresh, table, free, block, max(0, total - 5))  # dropped tokens
    run_plan(past, fresh, table, free[:need // 2], block, total)  # blocks run out
    run_plan(past, fresh, table[:, :2], free, block, total)       # the table is too narrow


def test_plan_edges():
    block = 16
    none = np.zeros((0, 4), np.int32)
    run_plan([], [], none, [5, 6], block, 0)
    run_plan([], [], none, [5, 6], block, 9)
    run_plan([0, 0], [0, 0], np.full((2, 3), -1, np.int32), [], block, 3)
    run_plan([-4, 3], [2, -7], np.array([[-1, -1], [9, -1]], np.int32), [1, 2], block, 4)   # negative lengths count as 0
    run_plan([3, 3], [2, 2], np.array([[-1, -1], [9, -1]], np.int32), [1, 2], block, 4)     # a held block is missing
    run_plan([5], [6], np.array([[2 ** 27]], np.int32), [1], block, 6)                      # slots above 2^31 - 1
    run_plan([2 ** 31 - 3], [6], np.array([[4]], np.int32), [1], block, 6)                  # positions above it
    run_plan([0, 4], [20, 2], np.full((2, 0), -1, np.int32), [7, 8], block, 22)             # a table without columns


def test_plan_huge_request_counts_are_saturated():
    got = qw.kv_plan(ints([0, 0, 0]), ints([2 ** 31 - 1] * 3), ints(np.full((3, 2), -1)), ints([7, 8, 9]), 16, 40)
    assert host(got.counts).tolist() == [2, 2 ** 31 - 1] and host(got.cu_tokens).tolist() == [0, 40, 40, 40]
    assert host(got.slots)[:33].tolist() == list(range(112, 128)) + list(range(128, 144)) + [-1]


# ---------------------------------------------------------------------------
# qk_norm_rope
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,pairs,norm", [
    (1, 1, 1, 64, 64, False, True), (1, 32, 2, 128, 64, True, False), (5, 7, 3, 128, 128, False, True),
    (33, 4, 2, 64, 32, True, True), (3, 2, 1, 128, 16, False, True), (2, 3, 3, 128, 0, True, True),
    (17, 5, 1, 64, 48, False, False), (9, 28, 4, 128, 96, False, True), (300, 16, 16, 64, 64, True, True),
])
def test_norm_rope(tokens, hq, hk, dim, rot, pairs, norm, dtype):
    say("norm_rope T=%d %d/%d D=%d rot=%d pairs=%s norm=%s %s" % (tokens, hq, hk, dim, rot, pairs, norm, dtype))
    rng = np.random.default_rng(tokens + dim + rot)
    span = 50
    qkv = dev(rng.standard_normal((tokens, (hq + 2 * hk) * dim)), dtype)
    q, k = qkv[:, :hq * dim].view(tokens, hq, dim), qkv[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    pos = rng.integers(0, span, tokens)
    if tokens > 2:
        pos[1], pos[2] = -1, span   # padding, and beyond the table
    angle = rng.uniform(0, 7, (span, rot // 2))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    wq, wk = (dev(1 + 0.3 * rng.standard_normal(dim), dtype) for _ in range(2)) if norm else (None, None)
    q0, k0 = host(q), host(k)
    got = qw.qk_norm_rope(q, k, ints(pos), dev(cos), dev(sin), wq, wk, eps=1e-5, interleaved=pairs)
    for g, x, w in zip(got, (q0, k0), (wq, wk)):
        want, mag = ref.norm_rope(x, pos, cos, sin, None if w is None else host(w), 1e-5, pairs)
        # one rounding to the type; the norm's sum and root and the rotation: dim + 8 fp32 roundings
        tol = unit(dtype) * np.abs(want) + (dim + 8) * 2.0 ** -24 * mag + 2.0 ** -25
        within(host(g), want, tol)
    # in place, on the fused tensor's columns: the same bits, and the values untouched
    v0 = qkv[:, (hq + hk) * dim:].clone()
    qw.qk_norm_rope(q, k, ints(pos), dev(cos), dev(sin), wq, wk, eps=1e-5, interleaved=pairs, out=(q, k))
    torch.cuda.synchronize()
    assert torch.equal(q, got[0]) and torch.equal(k, got[1]) and torch.equal(qkv[:, (hq + hk) * dim:], v0)


def test_norm_rope_zero_rows_and_no_tokens():
    q = torch.zeros((2, 2, 64), dtype=F16, device="cuda:0")
    k = torch.zeros((2, 1, 64), dtype=F16, device="cuda:0")
    one = torch.ones(64, dtype=F16, device="cuda:0")
    cos = torch.ones((4, 32), device="cuda:0")
    a, b = qw.qk_norm_rope(q, k, ints([0, 3]), cos, cos, one, one, eps=1e-6)
    assert not host(a).any() and not host(b).any()
    a, b = qw.qk_norm_rope(q[:0], k[:0], ints([]), cos, cos, one, one)
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)


# ---------------------------------------------------------------------------
# kv_write, kv_read
# ---------------------------------------------------------------------------

def write_and_compare(rng, slots, kv, dim, block, blocks, dtype, scale=1.0, cache=None, x=None):
    T = len(slots)
    if x is None:
        x = [dev(rng.standard_normal((T, kv, dim)) * scale * 2.0 ** rng.uniform(-3, 3, (T, 1, 1)), dtype) for _ in range(2)]
    cache = ref.random_cache(rng, blocks, kv, dim, block) if cache is None else cache
    on = [dev(c) for c in cache]
    say("write T=%d kv=%d D=%d B=%d %s" % (T, kv, dim, block, dtype))
    qw.kv_write(x[0], x[1], ints(slots), *on)
    k, ks = ref.write(host(x[0]), slots, cache[0], cache[2], False)
    v, vs = ref.write(host(x[1]), slots, cache[1], cache[3], True)
    # bit-exact, and nothing else in the cache has moved
    same(on[2].cpu().numpy(), ks, "key scales")
    same(on[3].cpu().numpy(), vs, "value scales")
    same(host(on[0]), k, "key codes")
    same(host(on[1]), v, "value codes")
    return (k, v, ks, vs), on


def slots_of(table, r, lo, hi, block):
    return [int(table[r, p // block]) * block + p % block for p in range(lo, hi)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("kv,dim", [(1, 64), (3, 128), (2, 128), (5, 64)])
def test_write_ragged(kv, dim, block, dtype):
    rng = np.random.default_rng(block + kv)
    past = [0, block - 1, 5, block, 0, 3 * block + 7, 1, 0]
    fresh = [1, 1, 3 * block + 2, 2, block, 1, 0, 2 * block + 1]
    context = [p + n for p, n in zip(past, fresh)]
    table, blocks = ref.pages(rng, context, block)
    slots = [s for r in range(len(past)) for s in slots_of(table, r, past[r], context[r], block)]
    # padding, and slots outside the cache, before, between (after the second request) and behind
    slots = [-1] + slots[:2] + [-1, blocks * block, 2 ** 31 - 1] + slots[2:] + [-1]
    write_and_compare(rng, slots, kv, dim, block, blocks, dtype)


def test_write_prompt_windows():
    """More tokens than the one-token-a-workgroup form takes, single tokens
    among them, runs that begin and end anywhere in a window."""
    rng = np.random.default_rng(5)
    block, kv, dim = 32, 2, 64
    fresh = [1] * 23 + [777] + [1] * 5 + [900, 13, 601] + [2] * 9
    past = [int(x) for x in rng.integers(0, 70, len(fresh))]
    context = [p + n for p, n in zip(past, fresh)]
    table, blocks = ref.pages(rng, context, block)
    slots = [s for r in range(len(past)) for s in slots_of(table, r, past[r], context[r], block)]
    assert len(slots) > 2048
    write_and_compare(rng, slots, kv, dim, block, blocks, F16)


@pytest.mark.parametrize("block", [16, 64, 128])
def test_write_token_by_token(block):
    """A block filled by one-token calls, its scale growing on the way, then
    started afresh."""
    rng = np.random.default_rng(block)
    cache = None
    for p in list(range(block)) + [0, 1]:
        grow = 2.0 ** (8.0 * p / block)
        cache, _ = write_and_compare(rng, [2 * block + p], 2, 64, block, 4, F16, scale=grow, cache=cache)


@pytest.mark.parametrize("dtype", TYPES)
def test_write_zero_tiny_and_large(dtype):
    rng = np.random.default_rng(3)
    block, kv, dim = 16, 2, 64
    big = 60000.0 if dtype == F16 else 3e38
    tiny = 6e-8 if dtype == F16 else 1e-38
    cache = tuple(np.zeros_like(c) for c in ref.random_cache(rng, 3, kv, dim, block))
    for p, size in enumerate([0.0, tiny, 1.0, 0.0, big, tiny, 1.0]):
        x = [dev(np.full((1, kv, dim), size) * rng.choice([-1, 1], (1, kv, dim)), dtype) for _ in range(2)]
        cache, on = write_and_compare(rng, [block + p], kv, dim, block, 3, dtype, cache=cache, x=x)


def test_write_ties_and_extremes():
    """x / S on half-integers exactly: a scale of 2^-3 and multiples of 2^-4."""
    x = (np.arange(-127, 128)[:, None] * np.ones(64) * 2.0 ** -4).reshape(255, 1, 64)[:128]
    x[0] = 127 * 2.0 ** -3
    t = dev(x, F16)
    cache = tuple(np.zeros_like(c) for c in ref.random_cache(np.random.default_rng(0), 2, 1, 64, 128))
    (k, _, ks, _), _ = write_and_compare(None, list(range(128)), 1, 64, 128, 2, F16, cache=cache, x=[t, t])
    assert ks[0, 0] == 2.0 ** -3 and np.array_equal(k[0, 0, 1:, 0], np.rint(np.arange(-126, 1) / 2.0))


def test_write_strided_inputs_and_empty():
    rng = np.random.default_rng(8)
    kv, dim, block, T = 2, 128, 64, 70
    fused = dev(rng.standard_normal((T, (4 + 2 * kv) * dim)), F16)
    k, v = fused[:, 4 * dim:(4 + kv) * dim].view(T, kv, dim), fused[:, (4 + kv) * dim:].view(T, kv, dim)
    write_and_compare(rng, list(range(64, 64 + T)), kv, dim, block, 4, F16, x=[k, v])
    write_and_compare(rng, [], kv, dim, block, 4, F16, x=[k[:0], v[:0]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,kv,dim", [(1, 1, 64), (63, 2, 128), (130, 3, 64), (200, 2, 128)])
def test_read(tokens, kv, dim, block, dtype):
    say("read T=%d kv=%d D=%d B=%d %s" % (tokens, kv, dim, block, dtype))
    rng = np.random.default_rng(tokens + block)
    blocks = -(-200 // block) + 2
    cache = ref.random_cache(rng, blocks, kv, dim, block)
    slots = np.arange(tokens) + 3                               # consecutive
    slots[tokens // 2:] = rng.integers(0, blocks * block, tokens - tokens // 2)
    if tokens > 3:
        slots[1], slots[3] = -1, blocks * block
    k, v = qw.kv_read(ints(slots), *[dev(c) for c in cache], dtype=dtype)
    for got, codes, scales, tr in ((k, cache[0], cache[2], False), (v, cache[1], cache[3], True)):
        want = ref.gather(slots, codes, scales, tr)
        exact = torch.from_numpy(want.astype(np.float32)).to(dtype).double().numpy()  # code * scale in fp32, then one rounding
        same(host(got), exact, "read")


# ---------------------------------------------------------------------------
# kv_attention
# ---------------------------------------------------------------------------

def compare_attention(rng, new, context, heads, kv, dim, block, dtype, causal=True, window=0, scale=None, q=None, cache=None,
                      table=None, max_new=None, max_context=None, spread=1.0):
    new, context = list(new), list(context)
    say("attention new=%s ctx=%s %d/%d D=%d B=%d %s causal=%s window=%d" % (new[:9], context[:9], heads, kv, dim, block, dtype,
                                                                        causal, window))
    made, blocks = ref.pages(rng, context, block)
    table = made if table is None else table
    cache = ref.random_cache(rng, blocks, kv, dim, block, spread) if cache is None else cache
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    q = dev(rng.standard_normal((T, heads, dim)) * 1.5, dtype) if q is None else q
    most = max(new) if max_new is None else max_new
    out = torch.full((T, heads, dim), float("nan"), dtype=dtype, device="cuda:0")
    got = qw.kv_attention(q, *[dev(c) for c in cache], ints(table), ints(context), ints(cu), most, max_context=max_context,
                          scale=scale, causal=causal, window=window, out=out)
    real = dim ** -0.5 if scale is None else scale
    want, mass, reach, tail = ref.attention(host(q), cache, table, context, cu, most, real, causal, window)
    within(host(got), want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(dtype)))
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (4, 4, 128), (32, 2, 128), (6, 2, 64), (28, 4, 128), (40, 1, 64)])
def test_attention_decode(heads, kv, dim, block, dtype):
    rng = np.random.default_rng(heads + block)
    compare_attention(rng, [1] * 7, [1, 0, block, block + 1, 63, 130, 517], heads, kv, dim, block, dtype)


@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("ctx", [255, 256, 257, 511, 513, 1500, 4097])
def test_attention_split_edges(ctx, block):
    compare_attention(np.random.default_rng(ctx), [1, 1, 1], [ctx, 3, ctx // 2], 8, 2, 64, block, F16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv,dim", [(2, 2, 64), (8, 2, 128), (9, 3, 64)])
def test_attention_prompt(heads, kv, dim, block, dtype):
    rng = np.random.default_rng(dim + block)
    new = [1, 70, 0, 129, 200]
    compare_attention(rng, new, new, heads, kv, dim, block, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 15, 64, 100])
@pytest.mark.parametrize("block", [16, 64])
def test_attention_chunk_and_windows(block, window, causal):
    rng = np.random.default_rng(block + window)
    compare_attention(rng, [5, 33, 100, 2], [300, 33, 700, 1], 4, 2, 64, block, F16, causal=causal, window=window)


@pytest.mark.parametrize("new", [2, 5, 8, 17])
def test_attention_drafts(new):
    compare_attention(np.random.default_rng(new), [new] * 3, [1000, new, 77], 8, 2, 128, 32, BF16)


def test_attention_rows_that_see_nothing():
    """More queries than cached tokens (their positions are negative), an idle
    request, and a request whose blocks are all missing."""
    rng = np.random.default_rng(1)
    new, context = [9, 1, 4, 80], [3, 0, 40, 20]
    table, blocks = ref.pages(rng, context, 16)
    table[2, :] = [-1] * table.shape[1]
    cache = ref.random_cache(rng, blocks, 2, 64, 16)
    got = host(compare_attention(rng, new, context, 4, 2, 64, 16, F16, table=table, cache=cache))
    assert not got[:6].any() and got[6:9].any() and not got[9:14].any()


def test_attention_missing_blocks_in_the_middle():
    rng = np.random.default_rng(2)
    context = [200, 90]
    table, blocks = ref.pages(rng, context, 16)
    table[0, 3], table[0, 7], table[1, 0] = -1, blocks, 2 ** 31 - 1
    compare_attention(rng, [1, 2], context, 4, 2, 64, 16, F16, table=table, cache=ref.random_cache(rng, blocks, 2, 64, 16))
    compare_attention(rng, [40, 2], context, 4, 2, 64, 16, F16, table=table, cache=ref.random_cache(rng, blocks, 2, 64, 16))


@pytest.mark.parametrize("new", [1, 40])
def test_attention_scales_far_apart(new):
    """Value scales over 2^40, and blocks of zeros (scale 0): the weights of
    one sum must not be lost against another block's scale."""
    rng = np.random.default_rng(new)
    context = [400, 150]
    table, blocks = ref.pages(rng, context, 16)
    k, v, ks, vs = ref.random_cache(rng, blocks, 2, 64, 16)
    ks *= np.float32(2.0 ** -4)
    vs *= (2.0 ** rng.uniform(-20, 0, vs.shape)).astype(np.float32)
    dead = table[0, [2, 5, 6]]
    vs[dead], v[dead] = 0, 0
    ks[table[0, 9]], k[table[0, 9]] = 0, 0
    compare_attention(rng, [new, new], context, 4, 2, 64, 16, BF16, cache=(k, v, ks, vs), table=table)
    vs[:], v[:] = 0, 0
    assert not host(compare_attention(rng, [new, new], context, 4, 2, 64, 16, F16, cache=(k, v, ks, vs), table=table)).any()


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("dtype", TYPES)
def test_attention_peaked_and_flat(new, dtype):
    """Scores in the hundreds (one key takes all, the reference maximum moves
    often) and scores of zero."""
    rng = np.random.default_rng(7)
    for gain in (40.0, 0.0):
        q = dev(rng.standard_normal((2 * new, 4, 64)) * gain, dtype)
        compare_attention(rng, [new, new], [333, 64 + new], 4, 2, 64, 64, dtype, q=q)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_bf16_range(new):
    """bf16 queries far outside fp16's range, against keys that bring the
    scores back."""
    rng = np.random.default_rng(11)
    for power in (-60, 60):
        q = dev(rng.standard_normal((new, 2, 64)) * 2.0 ** power, BF16)
        table, blocks = ref.pages(rng, [200], 32)
        k, v, ks, vs = ref.random_cache(rng, blocks, 1, 64, 32)
        compare_attention(rng, [new], [200], 2, 1, 64, 32, BF16, q=q, table=table,
                          cache=(k, v, (ks * 2.0 ** -power).astype(np.float32), vs))


@pytest.mark.parametrize("new", [1, 50])
def test_attention_hidden_garbage(new):
    """What a row does not see does not touch it: NaN and infinite scales in
    blocks of other requests, -128 codes behind the context's end."""
    rng = np.random.default_rng(13)
    context = [70, 129]
    table, blocks = ref.pages(rng, context, 64, spare=4)
    k, v, ks, vs = ref.random_cache(rng, blocks, 2, 64, 64)
    used = set(table[table >= 0].tolist())
    for b in range(blocks):
        if b not in used:
            ks[b], vs[b] = np.nan, np.inf
    k[table[0, 1], :, 6:], v[table[0, 1], :, :, 6:] = -128, -128
    compare_attention(rng, [new, new], context, 4, 2, 64, 64, F16, cache=(k, v, ks, vs), table=table)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_nan_and_inf_queries_stay_in_their_row(new):
    rng = np.random.default_rng(17)
    q = rng.standard_normal((new + 1, 2, 64))
    clean = dev(q, F16)
    q[0, 1, 5], q[-1, 0, 0] = np.nan, np.inf
    dirty = dev(q, F16)
    context, cu = [150 + new, 90], [0, new, new + 1]
    table, blocks = ref.pages(rng, context, 32)
    cache = [dev(c) for c in ref.random_cache(rng, blocks, 2, 64, 32)]
    say("attention with NaN queries, new=%d" % new)
    a, b = (host(qw.kv_attention(x, *cache, ints(table), ints(context), ints(cu), new)) for x in (clean, dirty))
    assert np.isnan(b[0, 1]).all() and np.isnan(b[-1, 0]).all()
    keep = np.ones(b.shape[:2], bool)
    keep[0, 1] = keep[-1, 0] = False
    assert np.array_equal(a[keep], b[keep])


def test_attention_scale_signs_and_zero():
    rng = np.random.default_rng(19)
    for scale in (0.0, -0.1, 0.3):
        compare_attention(rng, [1, 20], [100, 300], 4, 2, 64, 32, F16, scale=scale)


def test_attention_strided_queries_and_bounds():
    rng = np.random.default_rng(23)
    T, heads, kv, dim, block = 6, 4, 2, 64, 16
    fused = dev(rng.standard_normal((T, (heads + 2 * kv) * dim)), F16)
    q = fused[:, :heads * dim].view(T, heads, dim)
    a = compare_attention(rng, [4, 2], [40, 90], heads, kv, dim, block, F16, q=q)
    # a context beyond the table's width is taken as the width; max_context bounds it too
    context, cu = [33, 50], [0, 4, 6]
    table, blocks = ref.pages(rng, context, block)
    cache = ref.random_cache(rng, blocks, kv, dim, block)
    on = [dev(c) for c in cache]
    wide = table.shape[1] * block
    say("attention bounds")
    x = host(qw.kv_attention(q, *on, ints(table), ints([33, 10 ** 6]), ints(cu), 4))
    want, mass, reach, tail = ref.attention(host(q), cache, table, [33, wide], cu, 4, dim ** -0.5)
    within(x, want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(F16)))
    y = host(qw.kv_attention(q, *on, ints(table), ints([33, 50]), ints(cu), 4, max_context=37))
    want, mass, reach, tail = ref.attention(host(q), cache, table, [33, 37], cu, 4, dim ** -0.5)
    within(y, want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(F16)))
    assert a.shape == (T, heads, dim)


def test_attention_rows_of_no_request_are_left():
    rng = np.random.default_rng(29)
    table, blocks = ref.pages(rng, [40], 16)
    on = [dev(c) for c in ref.random_cache(rng, blocks, 1, 64, 16)]
    q = dev(rng.standard_normal((9, 2, 64)), F16)
    out = torch.full((9, 2, 64), 7.0, dtype=F16, device="cuda:0")
    qw.kv_attention(q, *on, ints(table), ints([40]), ints([2, 5]), 3, out=out)
    got = host(out)
    assert (got[:2] == 7).all() and (got[5:] == 7).all() and not (got[2:5] == 7).any()
    # offsets that are no such offsets stay inside the tensors
    qw.kv_attention(q, *on, ints(table), ints([40]), ints([-5, 10 ** 9]), 4, out=out)
    qw.kv_attention(q, *on, ints(table), ints([-40]), ints([8, 2]), 4, out=out)
    torch.cuda.synchronize()


def test_attention_is_deterministic_and_stream_ordered():
    """The same bits on every call, on another stream than the operands', and
    with a workspace of the caller's."""
    rng = np.random.default_rng(31)
    context, new = [3000, 1700, 64], [1, 1, 1]
    table, blocks = ref.pages(rng, context, 64)
    on = [dev(c) for c in ref.random_cache(rng, blocks, 2, 128, 64)]
    q = dev(rng.standard_normal((3, 32, 128)), F16)
    args = (q, *on, ints(table), ints(context), ints([0, 1, 2, 3]), 1)
    say("attention twice, and on another stream")
    first = qw.kv_attention(*args)
    n = qw.kv_attention_workspace(q, on[0], args[5], 1)
    assert n > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda:0")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = qw.kv_attention(*args, workspace=ws)
    third = qw.kv_attention(*args)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_long_cache_offsets():
    """A block whose codes begin beyond 2^32 bytes of the cache, and one
    beyond 2^31: written, read and attended to."""
    block, kv, dim = 128, 16, 128
    blocks = (2 ** 32 + 2 ** 20) // (block * kv * dim)
    say("cache of %d blocks, %.1f GiB a side" % (blocks, blocks * block * kv * dim / 2 ** 30))
    cache = qw.kv_cache(blocks, kv, dim, block)
    rng = np.random.default_rng(37)
    far, mid = blocks - 1, 2 ** 31 // (block * kv * dim) + 1
    x = [dev(rng.standard_normal((6, kv, dim)), F16) for _ in range(2)]
    slots = [far * block + 1, far * block + 2, mid * block, mid * block + 1, mid * block + 2, mid * block + 3]
    qw.kv_write(x[0], x[1], ints(slots), *cache)
    k, v = qw.kv_read(ints(slots), *cache)
    small = ref.random_cache(rng, 2, kv, dim, block)
    for c in small:
        c[:] = 0
    near = [1, 2, block, block + 1, block + 2, block + 3]
    kc, ks = ref.write(host(x[0]), near, small[0], small[2], False)
    vc, vs = ref.write(host(x[1]), near, small[1], small[3], True)
    assert np.array_equal(host(k), ref.gather(near, kc, ks, False).astype(np.float32).astype(np.float16).astype(np.float64))
    assert np.array_equal(host(v), ref.gather(near, vc, vs, True).astype(np.float32).astype(np.float16).astype(np.float64))
    q = dev(rng.standard_normal((2, kv, dim)), F16)
    got = host(qw.kv_attention(q, *cache, ints([[far], [mid]]), ints([3, 4]), ints([0, 1, 2]), 1))
    want, mass, reach, tail = ref.attention(host(q), (kc, vc, ks, vs), np.array([[0], [1]]), [3, 4], [0, 1, 2], 1, dim ** -0.5)
    within(got, want, ref.attention_tolerance(want, mass, reach, tail, dim, unit(F16)))
    del cache, k, v
    torch.cuda.empty_cache()
