"""route_experts where scores are so small that binary64 holds them as
subnormal numbers: they still have an order and shares."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F32 = torch.float32
GPU = "cuda:0"


def logits(seed, tokens, experts):
    """Between -712 and -704: exp() of them is from 6e-310 on, so more than 2^40
    steps of 2^-1074, and rounding to these is below 2^-40 relative."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    return -712 + torch.rand(tokens, experts, generator=gen).argsort(1).float() * (8.0 / experts)


def want(x, top_k, allowed):
    """ids by the logits among `allowed`, and each one's exp() over their sum."""
    ids, weights = [], []
    for row in x.double().tolist():
        best = sorted(allowed, key=lambda i: -row[i])[:top_k]
        s = [math.exp(row[i]) for i in best]  # (1 + exp(l) is 1 in binary64)
        ids.append(best)
        weights.append([v / sum(s) for v in s])
    return ids, torch.tensor(weights, dtype=torch.float64)


def assert_route(r, ids, weights):
    assert r.ids.tolist() == ids
    # fp64 to fp32: half a step of 2^-24; the scores' own errors are far below
    assert ((r.weights.cpu().double() - weights).abs() <= 1.01 * 2.0 ** -24 * weights).all()


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,top_k", [(16, 4), (128, 8), (256, 8), (512, 16)])
def test_sigmoid(experts, top_k, with_bias):
    x = logits(1, 30, experts)
    bias = torch.zeros(experts, device=GPU) if with_bias else None
    print("sigmoid", experts, top_k, with_bias, flush=True)
    assert_route(qw.route_experts(x.to(GPU), top_k, "sigmoid", bias=bias), *want(x, top_k, range(experts)))
    r = qw.route_experts(x.to(GPU), top_k, "sigmoid", bias=bias, renormalize=False)
    assert not r.weights.any()  # (below binary32's range)


@pytest.mark.parametrize("experts,top_k", [(16, 4), (256, 8)])
def test_softmax_whose_largest_is_not_chosen(experts, top_k):
    x = logits(2, 30, experts)
    x[:, 3] = 0.0
    bias = torch.zeros(experts)
    bias[3] = -2.0
    print("softmax", experts, top_k, flush=True)
    r = qw.route_experts(x.to(GPU), top_k, "softmax", bias=bias.to(GPU))
    assert_route(r, *want(x, top_k, [e for e in range(experts) if e != 3]))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_scores_that_are_zero(scoring):
    """Beyond binary64's range: no weight, and the order of the logits, or with a
    bias of the indexes."""
    x = torch.full((5, 24), -2000.0, device=GPU)
    x[:, 7:10] = -1000.0
    x[:, 2] = 0.0
    out = torch.zeros(24, device=GPU)
    out[2] = -math.inf
    r = qw.route_experts(x, 4, scoring, bias=out)
    assert r.ids.tolist() == [[0, 1, 3, 4]] * 5 and not r.weights.any()
    r = qw.route_experts(x, 4, scoring)
    assert r.ids.tolist() == [[2, 7, 8, 9]] * 5 and r.weights.tolist() == [[1.0, 0.0, 0.0, 0.0]] * 5


@pytest.mark.parametrize("scale", [0.1, 2.446, 1e39, -3.0, 1e-41, 0.0])
def test_scale(scale):
    """A factor that binary32 does not hold, or not exactly, counts as it is: one
    rounding to 32 bits, that of the weight."""
    gen = torch.Generator()
    gen.manual_seed(3)
    x = torch.randn(400, 64, generator=gen)
    x[:, 8:] = -1e4  # (not chosen)
    r = qw.route_experts(x.to(GPU), 8, "sigmoid", renormalize=False, scale=scale)
    w = torch.sigmoid(x.double()).gather(1, r.ids.long().cpu()) * scale
    got = r.weights.cpu().double()
    inf = w.abs() > torch.finfo(F32).max
    assert torch.equal(got.isinf(), inf) and (not inf.any() or scale > 1e38)
    # half a step of 2^-24, or of the subnormal numbers' 2^-149
    assert ((got - w).abs() <= 1.01 * 2.0 ** -24 * w.abs() + 2.0 ** -150)[~inf].all()
