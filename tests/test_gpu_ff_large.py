"""The feed-forward calls where an operand is longer than 2^32 bytes or 2^31
elements: rows of its beginning, middle and end."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import assert_rounded, linear64  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16, I8, I32 = torch.float16, torch.int8, torch.int32
GPU = "cuda:0"


def say(*what):
    print(*what, flush=True)


def some(count):
    return torch.tensor(sorted({0, 1, count // 3, count // 2 + 7, count - 2, count - 1}), device=GPU)


def ints(seed, shape, top, dtype):
    g = torch.Generator(device=GPU)
    g.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=GPU, dtype=I8).to(dtype)


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.get_device_properties(0).total_memory < (64 << 30):
        pytest.skip("needs 64 GiB")
    yield
    torch.cuda.empty_cache()


def test_norm():
    T, K = 140000, 16384
    say("norm", T, K)
    x, r = ints(1, (T, K), 100, F16), ints(2, (T, K), 100, F16)
    w = torch.ones(K, dtype=F16, device=GPU)
    y, h = qw.add_rms_norm(x, w, residual=r, out=(None, x.clone()))
    at = some(T)
    want = (x[at].double() + r[at].double())
    assert torch.equal(h[at].double(), want)
    y64 = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert_rounded(y[at], y64, 2.0 ** -20 * y64.abs())
    del y
    q, s, h = qw.add_rms_norm(x, w, residual=r, quantize=True, out=(None, None, x))
    assert torch.equal(h[at].double(), want)
    assert ((q[at].double() * s[at].double()[:, None] - y64).abs() <= 0.51 * s[at].double()[:, None] + 2.0 ** -10 * y64.abs()).all()


@pytest.mark.parametrize("gated", [False, True])
def test_linear_rows(gated):
    m, n, k = 600000, 4096, 4096
    say("linear", m, n, k, gated)
    x, q = ints(3, (m, k), 3, F16), ints(4, (n, k), 127, I8)
    s = torch.full((n,), 2.0 ** -12, dtype=F16, device=GPU)
    y = qw.w8a16_linear(x, q, s, activation="relu", gated=gated)
    at = some(m)
    assert_rounded(y[at], *linear64(x[at], q, s, None, "relu", gated))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [2, 12, 200])
def test_linear_channels(m, gated):
    """A weight of more than 2^32 bytes (gated by the skinny kernel beyond the
    MFMA kernels' range)."""
    n, k = 600064, 8192
    say("linear", m, n, k, gated)
    x, q = ints(5, (m, k), 3, F16), ints(6, (n, k), 127, I8)
    s = torch.full((n,), 2.0 ** -12, dtype=F16, device=GPU)
    y = qw.w8a16_linear(x, q, s, gated=gated)
    at = some(n // 2 if gated else n)
    rows = torch.cat((at, at + n // 2)) if gated else at
    assert_rounded(y[:, at], *linear64(x, q[rows], s[rows], None, None, gated))


@pytest.mark.parametrize("tokens", [40, 3000])
def test_experts_weights(tokens):
    E, n, k, top = 96, 8192, 8192, 2
    say("experts", tokens, E, n, k)
    q = ints(7, (E, n, k), 127, I8)
    s = torch.full((E, n), 2.0 ** -12, dtype=F16, device=GPU)
    x = ints(8, (tokens, k), 3, F16)
    g = torch.Generator(device=GPU)
    g.manual_seed(9)
    route = qw.route_experts(torch.randn(tokens, E, generator=g, device=GPU), top)
    y = qw.w8a16_experts(x, q, s, route)
    offsets, rows = route.offsets.tolist(), route.rows.long()
    for e in (0, 1, E // 2, E - 2, E - 1):
        if offsets[e] < offsets[e + 1]:
            at = torch.arange(offsets[e], offsets[e + 1], device=GPU)[:20]
            assert_rounded(y[at], *linear64(x[rows[at] // top], q[e], s[e]))


def test_experts_rows():
    """Outputs and inputs (in the route's order) of more than 2^32 bytes."""
    tokens, E, top, n, k = 150000, 8, 8, 4096, 2048
    say("experts", tokens, E, n, k)
    route = qw.route_experts(torch.zeros(tokens, E, device=GPU), top)
    assert route.offsets.tolist() == [e * tokens for e in range(E + 1)]
    x, q = ints(10, (tokens * top, k), 3, F16), ints(11, (E, n, k), 127, I8)
    s = torch.full((E, n), 2.0 ** -12, dtype=F16, device=GPU)
    y = qw.w8a16_experts(x, q, s, route, gather=False)
    for p in some(tokens * top).tolist():
        assert_rounded(y[p:p + 1], *linear64(x[p:p + 1], q[p // tokens], s[p // tokens]))
    out = qw.experts_combine(y, route)
    at = some(tokens)
    want = sum(y[at + e * tokens].double() for e in range(E)) / 8
    assert_rounded(out[at], want, 2.0 ** -20 * sum(y[at + e * tokens].double().abs() for e in range(E)))
