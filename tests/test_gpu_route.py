"""route_experts against plain Python in 64 bits: ids, list and weights."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import listing, route64  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def check(logits, top_k, bias=None, **more):
    print("route", tuple(logits.shape), logits.dtype, top_k, bias is not None, more, flush=True)
    r = qw.route_experts(logits, top_k, bias=bias, **more)
    ids, weights = route64(logits.cpu(), top_k, bias=None if bias is None else bias.cpu(), **more)
    assert r.ids.tolist() == ids
    offsets, rows, places = listing(ids, logits.shape[1])
    assert r.offsets.tolist() == offsets
    assert r.rows.tolist() == rows
    assert r.places.view(-1).tolist() == places
    want = torch.tensor(weights, dtype=torch.float64).view(logits.shape[0], top_k)
    got = r.weights.cpu().double()
    # fp64 to fp32: half a step of 2^-24; the oracle's own sums are exact beside it
    assert ((got - want).abs() <= 1.01 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all()
    return r


def normal(seed, tokens, experts, dtype=F32, size=1.5):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (size * torch.randn(tokens, experts, generator=gen, device="cuda")).to(dtype)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 8, 2), (3, 3, 3), (17, 60, 6), (64, 64, 8), (33, 65, 1), (5, 127, 4),
                                                  (300, 128, 8), (9, 160, 6), (16, 257, 10), (70, 512, 64), (2, 4, 9)])
def test_sizes(tokens, experts, top_k, dtype, scoring):
    check(normal(1, tokens, experts, dtype), top_k, scoring=scoring)
    check(normal(2, tokens, experts, dtype), top_k, scoring=scoring, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,top_k", [(8, 2), (64, 6), (100, 5), (256, 8), (512, 8)])
def test_bias(experts, top_k, scoring):
    bias = normal(3, 1, experts, size=0.05)[0]
    check(normal(4, 45, experts), top_k, bias=bias, scoring=scoring)
    check(normal(5, 45, experts, BF16), top_k, bias=bias, scoring=scoring, renormalize=False)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 64, 3, 2), (12, 4, 2, 4), (14, 2, 1, 7),
                                                             (6, 3, 1, 5), (512, 32, 5, 8), (16, 1, 1, 4), (16, 4, 4, 4)])
def test_groups(experts, groups, top_groups, top_k, with_bias):
    bias = normal(6, 1, experts, size=0.05)[0] if with_bias else None
    for scoring in ("softmax", "sigmoid"):
        check(normal(7, 37, experts), top_k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts", [8, 64, 160, 256])
def test_ties(experts, with_bias, groups):
    """Few different values, so that most choices are ties."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    logits = torch.randint(0, 3, (50, experts), generator=gen, device="cuda").to(F16)
    bias = torch.randint(0, 2, (experts,), generator=gen, device="cuda").float() / 8 if with_bias else None
    check(logits, 6, bias=bias, scoring="sigmoid", groups=groups, top_groups=max(1, groups // 2))
    check(torch.zeros(20, experts, device="cuda"), 4, bias=bias, groups=groups, top_groups=1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_logits_that_are_not_finite(scoring, with_bias):
    logits = normal(9, 24, 16)
    logits[0] = -INF
    logits[1] = NAN
    logits[2, :14] = -INF          # fewer than top_k left
    logits[3, 3:9] = NAN
    logits[4, 5] = INF
    logits[5, 5], logits[5, 6] = INF, INF
    logits[6] = torch.finfo(F32).min
    logits[7] = -200.0
    logits[8] = 300.0
    logits[9, :] = -INF
    logits[9, 15] = torch.finfo(F32).min
    bias = normal(10, 1, 16, size=0.05)[0] if with_bias else None
    check(logits, 4, bias=bias, scoring=scoring)
    check(logits, 4, bias=bias, scoring=scoring, renormalize=False)
    check(logits, 4, bias=bias, scoring=scoring, groups=4, top_groups=2)


def test_masked_experts():
    """A bias of -infinity takes an expert out."""
    bias = torch.zeros(32, device="cuda")
    bias[3:30] = -INF
    bias[31] = NAN
    r = check(normal(11, 20, 32), 6, bias=bias, scoring="sigmoid", renormalize=False)
    assert (r.ids[:, 4:] == -1).all()


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_large_biases(scoring, groups):
    """One of infinity puts an expert before all others, and the largest numbers
    lose the scores' bits and overflow as a group's sum, in fp32."""
    for values in ((INF, 0.0, INF, -INF), (3e38, 3e38, -3e38, 1e30), (INF, 3e38, NAN, -3e38)):
        bias = normal(15, 1, 32, size=0.05)[0]
        for i, v in enumerate(values):
            bias[5 + 7 * i] = v
        for top_k in (1, 2, 6):
            check(normal(16, 40, 32), top_k, bias=bias, scoring=scoring, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("groups", [1, 4])
def test_signed_zeros_tie(groups, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(17)
    x = torch.zeros(60, 64, dtype=dtype, device="cuda")
    x[torch.rand(x.shape, generator=gen, device="cuda") < 0.5] = -0.0
    x[::2, 10] = 1.0
    check(x, 5, groups=groups, top_groups=max(1, groups // 2))
    check(x, 5, scoring="sigmoid", groups=groups, top_groups=1)


@pytest.mark.parametrize("tokens", [1000, 4096, 4097, 9001])
def test_many_tokens(tokens):
    check(normal(12, tokens, 64, BF16), 4)


def test_every_token_to_one_expert():
    logits = torch.full((3000, 40), -INF, device="cuda")
    logits[:, 17] = 1.0
    r = check(logits, 1)
    assert r.offsets.tolist() == [0] * 18 + [3000] * 23


def test_close_choices():
    """Scores whose difference fp32 loses: the larger one in fp64 is taken."""
    x = torch.full((64, 8), -3.0, device="cuda")
    for t in range(64):
        x[t, t % 8] = -3.0 + 2.0 ** -21
    r = check(x, 1, bias=torch.ones(8, device="cuda"), scoring="sigmoid")
    assert r.ids.view(-1).tolist() == [t % 8 for t in range(64)]


def test_no_tokens():
    r = qw.route_experts(torch.empty(0, 24, device="cuda"), 3)
    assert r.ids.shape == (0, 3) and r.offsets.tolist() == [0] * 25 and r.rows.numel() == 0


def test_same_bits_again():
    x, b = normal(13, 2000, 128), normal(14, 1, 128, size=0.1)[0]
    a = qw.route_experts(x, 6, "sigmoid", bias=b, groups=8, top_groups=4)
    for _ in range(3):
        for u, v in zip(a, qw.route_experts(x, 6, "sigmoid", bias=b, groups=8, top_groups=4)):
            assert torch.equal(u, v)
