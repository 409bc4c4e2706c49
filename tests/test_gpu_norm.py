"""add_rms_norm against 64 bits."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import assert_rounded  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16, BF16 = torch.float16, torch.bfloat16
# The sum of squares is a tree over at most 64 terms a lane and 16 waves: 90
# roundings of 2^-24 relative at most, halved by the root; a few more follow.
OFF = 2.0 ** -18


def operands(seed, tokens, k, dtype, residual=True, size=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (size * torch.randn(tokens, k, generator=gen, device="cuda")).to(dtype)
    r = (5 * size * torch.randn(tokens, k, generator=gen, device="cuda")).to(dtype) if residual else None
    w = (1 + 0.3 * torch.randn(k, generator=gen, device="cuda")).to(dtype)
    return x, r, w


def norm64(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)  # (the fp32 sum of two 16-bit values rounds like the exact one)
    d = h.double()
    return h, d * w.double() / (d.square().mean(1, keepdim=True) + eps).sqrt()


def check(x, r, w, eps=1e-6, **more):
    print("norm", tuple(x.shape), x.dtype, r is not None, flush=True)
    h64, y64 = norm64(x, r, w, eps)
    y, h = qw.add_rms_norm(x, w, residual=r, eps=eps)
    assert torch.equal(h, h64)
    assert_rounded(y, y64, OFF * y64.abs())
    q, s, h = qw.add_rms_norm(x, w, residual=r, eps=eps, quantize=True)
    assert torch.equal(h, h64)
    check_codes(q, s, y64)


def check_codes(q, s, y64):
    bound = y64.abs().amax(1) / 127
    assert_rounded(s, bound, OFF * bound)
    scale = s.double()[:, None]
    units = torch.where(scale > 0, y64 / scale, 0.0)
    # half a step, and fp32's error of a quotient of at most 127.1
    near = (q.double() - units.clamp(-127, 127)).abs()
    assert (near <= 0.5 + 128 * 2 * OFF).all()
    assert q.min() >= -127


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("tokens,k", [(1, 16), (1, 4096), (3, 48), (5, 528), (8, 2064), (2, 8192), (33, 1024), (7, 16384), (2, 65536),
                                      (1, 32784), (2050, 512), (1100, 4096), (4099, 64)])
def test_sizes(tokens, k, dtype, residual):
    check(*operands(1, tokens, k, dtype, residual))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens", [3, 3000])
def test_small_and_large_rows(dtype, tokens):
    for size in (0.0, 1e-6, 1e3):
        check(*operands(2, tokens, 256, dtype, size=size))
    check(*operands(3, tokens, 256, dtype, size=1e-6), eps=0.0)
    x, r, w = operands(4, tokens, 256, dtype)
    check(x * 0, r * 0, w, eps=1e-6)  # rows of zeros: scale 0, codes 0
    q, s, _ = qw.add_rms_norm(x * 0, w, quantize=True)
    assert not q.any() and not s.any()


def test_zero_rows_without_eps():
    """0 / 0 is not asked for: eps 0 and a row of zeros give zeros or NaN of that
    row alone."""
    x, r, w = operands(5, 5, 128, F16)
    x[2] = 0
    r[2] = 0
    y, h = qw.add_rms_norm(x, w, residual=r, eps=0.0)
    _, want = norm64(x, r, w, 1e-30)
    keep = torch.tensor([0, 1, 3, 4], device="cuda")
    assert_rounded(y[keep], want[keep], OFF * want[keep].abs())


@pytest.mark.parametrize("tokens", [5, 2500])
def test_rows_that_are_not_finite_stay_alone(tokens):
    x, r, w = operands(6, tokens, 512, F16)
    want = qw.add_rms_norm(x, w, residual=r, quantize=True)
    x2 = x.clone()
    x2[1, 7] = float("nan")
    x2[3, 500] = float("inf")
    got = qw.add_rms_norm(x2, w, residual=r, quantize=True)
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[1] = keep[3] = False
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])


def test_strides_and_places():
    """Rows of wider matrices, and h in the place of either input."""
    for tokens in (6, 1500):
        x, r, w = operands(7, tokens, 256, BF16)
        want = qw.add_rms_norm(x, w, residual=r)
        wide = torch.zeros(tokens, 800, dtype=BF16, device="cuda")
        wide[:, 8:264], wide[:, 264:520] = x, r
        xs, rs = wide[:, 8:264], wide[:, 264:520]
        for a, b in zip(qw.add_rms_norm(xs, w, residual=rs), want):
            assert torch.equal(a, b)
        y, h = qw.add_rms_norm(xs, w, residual=rs, out=(None, rs))
        assert h is rs and torch.equal(rs, want[1]) and torch.equal(y, want[0])
        assert torch.equal(xs, x) and not wide[:, :8].any() and not wide[:, 520:].any()
        y, h = qw.add_rms_norm(x, w, residual=r, out=(torch.empty_like(x), x))
        assert h is x and torch.equal(x, want[1]) and torch.equal(y, want[0])


def test_no_tokens():
    x, r, w = operands(8, 0, 64, F16)
    y, h = qw.add_rms_norm(x, w, residual=r)
    assert y.shape == h.shape == (0, 64)


def test_feeds_the_product():
    x, r, w = operands(9, 40, 512, F16)
    q, s, h = qw.add_rms_norm(x, w, residual=r, quantize=True)
    qq, ss = qw.quantize_weights(torch.randn(96, 512, device="cuda") / 16)
    got = qw.w8a8_linear(q, s, qq, ss).double()
    _, y = norm64(x, r, w, 1e-6)
    want = y @ (qq.double() * ss.double()[:, None]).t()
    # a code is off by half a step of its row's scale: independent errors of
    # S / sqrt(12) over 512 products with weights of 1 / 16
    step = s.double()[:, None] / 12 ** 0.5 * 512 ** 0.5 / 16
    assert ((got - want).abs() <= 6 * step + 2.0 ** -10 * want.abs()).all()
