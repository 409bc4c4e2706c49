"""w8a16_experts and experts_combine against 64 bits, on every kernel and tile."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import assert_rounded, integers, linear64, made_route, scale16  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16 = torch.float16
TILES = [256256, 256128, 256064, 128064]


def ids_of(seed, tokens, experts, top_k, none=0.0, favourite=None):
    gen = torch.Generator()
    gen.manual_seed(seed)
    score = torch.rand(tokens, experts, generator=gen)
    if favourite is not None:
        score[:, favourite] += 1
    ids = score.topk(top_k, 1).indices
    ids[torch.rand(tokens, top_k, generator=gen) < none] = -1
    return ids.tolist()


def operands(seed, x_rows, experts, n, k, bias=True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = integers(gen, (x_rows, k), 4, F16)
    q = integers(gen, (experts, n, k), 127, torch.int8)
    s = scale16(gen, (experts, n), 2.0 ** -7 / k ** 0.5)
    return x, q, s, torch.randn(experts, n, generator=gen, device="cuda").half() if bias else None


def want_of(x, q, s, b, route, act, gated, gather):
    top_k = route.ids.shape[1]
    offsets, rows = route.offsets.tolist(), route.rows.long()
    y = torch.zeros(rows.numel(), q.shape[1] // (2 if gated else 1), dtype=torch.float64, device="cuda")
    off = torch.zeros_like(y)
    for e in range(q.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            src = x[rows[lo:hi] // top_k] if gather else x[lo:hi]
            y[lo:hi], off[lo:hi] = linear64(src, q[e], s[e], None if b is None else b[e], act, gated)
    return y, off


def check(seed, ids, experts, n, k, act=None, gated=False, gather=True, bias=True, path="auto", tile=0):
    print("experts", len(ids), "x", len(ids[0]), "of", experts, n, k, act, gated, gather, path, tile, flush=True)
    route = made_route(ids)(experts)
    entries, top_k = route.rows.numel(), len(ids[0])
    x, q, s, b = operands(seed, len(ids) if gather else entries, experts, n, k, bias)
    want, off = want_of(x, q, s, b, route, act, gated, gather)
    y = torch.full((entries, want.shape[1]), 55.0, dtype=F16, device="cuda")
    st = qw.library().qw_w8a16_experts_path(
        x.data_ptr(), x.shape[0], int(gather), q.data_ptr(), s.data_ptr(), None if b is None else b.data_ptr(),
        qw.ACTIVATIONS[act], int(gated), route.offsets.data_ptr(), route.rows.data_ptr(), entries, top_k, y.data_ptr(), experts,
        n, k, qw.PATHS[path], tile, torch.cuda.current_stream().cuda_stream)
    assert st == 0, qw.status_string(st)
    assert_rounded(y, want, off)
    assert not y[route.offsets[-1]:].any()
    return x, q, s, b, route, y


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 1, 1, 16, 16), (1, 8, 2, 64, 64), (7, 5, 3, 34, 48), (32, 64, 8, 130, 272),
                                                      (40, 3, 2, 256, 1040), (3, 512, 4, 32, 32), (64, 16, 1, 528, 128)])
def test_skinny(tokens, experts, top_k, n, k, gather, gated):
    check(1, ids_of(2, tokens, experts, top_k, none=0.2), experts, n, k, "silu", gated, gather, path="skinny")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tokens,experts,top_k,n,k,none", [(1, 2, 1, 2, 16, 0.0), (90, 4, 2, 260, 80, 0.1), (600, 3, 2, 518, 208, 0.3),
                                                           (257, 1, 1, 300, 64, 0.0), (700, 9, 4, 512, 400, 0.0)])
def test_tiles(tokens, experts, top_k, n, k, none, tile, gated):
    ids = ids_of(3, tokens, experts, top_k, none)
    check(4, ids, experts, n, k, "silu" if gated else "relu", gated, True, path="mfma", tile=tile)
    check(5, ids, experts, n, k, None, gated, False, bias=False, path="mfma", tile=tile)


@pytest.mark.parametrize("tokens", [1, 20, 333, 2000])
def test_auto(tokens):
    check(6, ids_of(7, tokens, 8, 3), 8, 192, 320, "gelu", False)
    check(8, ids_of(9, tokens, 8, 3, favourite=5), 8, 384, 320, "silu", True)


@pytest.mark.parametrize("path,tile", [("skinny", 0), ("mfma", 256256), ("mfma", 256064)])
def test_uneven_experts(path, tile):
    """All entries to the first, to the last, to none; ends on tile borders."""
    for ids in ([[0]] * 300, [[5]] * 300, [[-1]] * 300, [[0]] * 256 + [[3]] * 64 + [[5]] * 16 + [[-1]], [[2]] * 255 + [[3]] * 257,
                [[-1]] * 40 + [[1]] * 15 + [[2]] * 17):
        check(10, ids, 6, 64, 96, path=path, tile=tile)


@pytest.mark.parametrize("tile", [256256, 128064])
def test_odd_columns(tile):
    check(11, ids_of(12, 100, 3, 2), 3, 331, 96, "gelu", path="mfma", tile=tile)
    check(13, ids_of(14, 100, 3, 2), 3, 2 * 331, 96, "silu", True, path="mfma", tile=tile)
    check(15, ids_of(16, 9, 3, 2), 3, 331, 96, path="skinny")


@pytest.mark.parametrize("path,tile", [("skinny", 0), ("mfma", 256256), ("mfma", 128064)])
def test_same_expert_twice(path, tile):
    """A token may list an expert more than once."""
    check(17, [[1, 1, 2], [2, 2, 2], [0, 1, 0]] * 20, 3, 64, 64, path=path, tile=tile)


@pytest.mark.parametrize("path,tile", [("skinny", 0), ("mfma", 256256), ("mfma", 256128)])
def test_lists_that_are_not_routes(path, tile):
    """Indexes and offsets outside of what there is: rows of zeros, entries
    within the buffers."""
    x, q, s, b, route, y = check(18, ids_of(19, 50, 4, 2), 4, 64, 64, path=path, tile=tile)

    def run(offsets, rows):
        out = torch.full_like(y, 9.0)
        st = qw.library().qw_w8a16_experts_path(
            x.data_ptr(), 50, 1, q.data_ptr(), s.data_ptr(), b.data_ptr(), 0, 0, offsets.data_ptr(), rows.data_ptr(), 100, 2,
            out.data_ptr(), 4, 64, 64, qw.PATHS[path], tile, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        return out

    rows = route.rows.clone()
    rows[3], rows[60], rows[99] = -1, 100, 2 ** 31 - 1
    out = run(route.offsets, rows)
    e = torch.searchsorted(route.offsets[1:], torch.arange(100, device="cuda", dtype=torch.int32), right=True)
    for p in range(100):
        assert torch.equal(out[p], b[e[p]] if p in (3, 60, 99) else y[p])
    far = route.offsets.clone()
    far[0], far[-1] = -5, 2 ** 30
    assert torch.equal(run(far, route.rows), y)
    run(torch.tensor([90, 10, 200, -7, 50], dtype=torch.int32, device="cuda"), route.rows)  # (any values, but no fault)


def combine64(y, route, residual):
    places, w = route.places.long(), route.weights.double()
    each = torch.where((places < 0)[:, :, None], 0.0, y.double()[places.clamp(min=0)]) * w[:, :, None]
    total = each.sum(1)
    # one rounding of 2^-24 of the running sum for each term
    size = each.abs().sum(1)
    if residual is not None:
        total = total + residual.double()
        size = size + residual.double().abs()
    return total, 2.0 ** -24 * (places.shape[1] + 1) * size


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,n", [(1, 1, 1, 8), (1, 8, 2, 1), (5, 8, 8, 333), (64, 64, 6, 2048), (30, 100, 19, 40), (3000, 16, 2, 24)])
def test_combine(tokens, experts, top_k, n, residual):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(20)
    w = torch.rand(tokens, top_k, generator=gen, device="cuda")
    route = made_route(ids_of(21, tokens, experts, top_k, none=0.2), w)(experts)
    y = torch.randn(tokens * top_k, n, generator=gen, device="cuda").half()
    y[route.offsets[-1]:] = float("nan")  # (never read)
    r = torch.randn(tokens, n, generator=gen, device="cuda").half() if residual else None
    want, off = combine64(y, route, r)
    got = qw.experts_combine(y, route, residual=r)
    assert_rounded(got, want, off)
    if residual:
        assert qw.experts_combine(y, route, residual=r, out=r) is r
        assert torch.equal(r, got)


def test_tokens_of_no_expert():
    route = made_route([[-1, -1], [0, -1], [-1, -1]])(2)
    x, q, s, b = operands(22, 3, 2, 48, 32)
    y = qw.w8a16_experts(x, q, s, route, bias=b)
    r = torch.randn(3, 48, device="cuda").half()
    out = qw.experts_combine(y, route, residual=r)
    assert torch.equal(out[0], r[0]) and torch.equal(out[2], r[2]) and not torch.equal(out[1], r[1])
    assert not qw.experts_combine(y, route)[0].any()


def test_no_tokens():
    route = qw.route_experts(torch.empty(0, 4, device="cuda"), 2)
    x, q, s, b = operands(23, 0, 4, 64, 32)
    y = qw.w8a16_experts(x, q, s, route, bias=b)
    assert y.shape == (0, 64)
    assert qw.experts_combine(y, route).shape == (0, 64)


@pytest.mark.parametrize("tokens", [1, 12, 500])
def test_together(tokens):
    """Norm, router, both products and the sum, against the same in 64 bits from
    the values as they are rounded between the operators."""
    E, top_k, K, inner = 12, 3, 256, 192
    gen = torch.Generator(device="cuda")
    gen.manual_seed(24)
    x = torch.randn(tokens, K, generator=gen, device="cuda").half()
    stream = torch.randn(tokens, K, generator=gen, device="cuda").half()
    w = (1 + 0.1 * torch.randn(K, generator=gen, device="cuda")).half()
    up = [qw.quantize_weights(torch.randn(2 * inner, K, generator=gen, device="cuda") / K ** 0.5) for _ in range(E)]
    down = [qw.quantize_weights(torch.randn(K, inner, generator=gen, device="cuda") / inner ** 0.5) for _ in range(E)]
    up, down = ([torch.stack(t) for t in zip(*pairs)] for pairs in (up, down))
    router = torch.randn(E, K, generator=gen, device="cuda").half() / 16
    y, h = qw.add_rms_norm(x, w, residual=stream)
    route = qw.route_experts((y.float() @ router.float().t()), top_k)
    g = qw.w8a16_experts(y, *up, route, activation="silu", gated=True)
    d = qw.w8a16_experts(g, *down, route, gather=False)
    out = qw.experts_combine(d, route, residual=h)
    want_g, _ = want_of(y, *up, None, route, "silu", True, True)
    # the plain product's contract for each factor
    assert (g.double() - want_g).abs().max() <= 3 * (2e-3 * want_g.abs().max() + 1e-3)
    want_d, _ = want_of(g, *down, None, route, None, False, False)
    assert (d.double() - want_d).abs().max() <= 2e-3 * want_d.abs().max() + 1e-3
    want, off = combine64(d, route, h)
    assert_rounded(out, want, off)
