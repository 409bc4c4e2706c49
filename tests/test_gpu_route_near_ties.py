"""route_experts where fp64 numbers decide that agree in their upper words, in
every pair of lanes: groups and experts on the path of all in fp64."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F32 = torch.float32
GPU = "cuda:0"
INF = float("inf")


def route64(logits, top_k, scoring, bias, groups=1, top_groups=1):
    """ids of each token, in float64 (finite inputs, more experts than top_k)."""
    x = logits.double()
    s = 1 / (1 + torch.exp(-x)) if scoring == "sigmoid" else torch.softmax(x, 1)
    c = x if bias is None else s + bias.double()
    T, E = c.shape
    if groups > 1:
        by = c.view(T, groups, E // groups)
        score = by.amax(2) if bias is None else by.topk(2, dim=2).values.sum(2)
        first = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, first, True)
        c = torch.where(kept[:, :, None], by, -INF).view(T, E)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :top_k]
    w = s.gather(1, ids)
    return ids, w / w.sum(1, keepdim=True)


def pairs(count):
    """All ordered pairs of two different numbers below `count`, a row each."""
    a = torch.arange(count, device=GPU)
    p = torch.cartesian_prod(a, a)
    return p[p[:, 0] != p[:, 1]]


# experts and places for which a token has 16, 32 and 64 lanes (P experts each)
LANES = [(64, 2, 16, 4), (128, 8, 16, 8), (256, 8, 32, 8), (512, 8, 64, 8), (64, 40, 64, 8)]


@pytest.mark.parametrize("experts,groups", [(64, 8), (60, 4), (128, 16), (256, 8), (256, 32), (160, 20), (512, 64), (512, 16)])
def test_groups(experts, groups):
    """The scores of two groups are 1 and 1 + 2^-31: sigmoid(0) is 1/2, and its
    slope there 1/4."""
    print("groups", experts, groups, flush=True)
    size, p = experts // groups, pairs(groups)
    x = torch.full((len(p), experts), -4.0, device=GPU)
    t = torch.arange(len(p), device=GPU)
    for g in (0, 1):
        x[t, p[:, g] * size], x[t, p[:, g] * size + size - 1] = 0.0, 0.0
    x[t, p[:, 1] * size + size - 1] = 2.0 ** -29
    r = qw.route_experts(x, 2, "sigmoid", bias=torch.zeros(experts, device=GPU), groups=groups, top_groups=1)
    first = p[:, 1] * size
    assert torch.equal(r.ids.long(), torch.stack((first + size - 1, first), 1))
    # and with both groups: three experts tie behind the first
    r = qw.route_experts(x, 4, "sigmoid", bias=torch.zeros(experts, device=GPU), groups=groups, top_groups=2)
    tied = torch.stack((p[:, 0] * size, p[:, 0] * size + size - 1, first), 1).sort(1).values
    assert torch.equal(r.ids.long(), torch.cat(((first + size - 1)[:, None], tied), 1))


@pytest.mark.parametrize("experts,top_k,lanes,each", LANES)
def test_experts(experts, top_k, lanes, each):
    """Softmax with a bias: two experts of different lanes, exp(0) and exp(2^-31)
    over their sum; top_k reaches others below them."""
    print("experts", experts, top_k, flush=True)
    p = pairs(min(lanes, experts // each)) * each
    x = (torch.arange(experts, device=GPU, dtype=F32) * -0.01 - 4.0).repeat(len(p), 1)
    t = torch.arange(len(p), device=GPU)
    x[t, p[:, 0] + each // 2], x[t, p[:, 1]] = 0.0, 2.0 ** -31
    bias = torch.zeros(experts, device=GPU)
    r = qw.route_experts(x, top_k, "softmax", bias=bias)
    assert torch.equal(r.ids[:, :2].long(), torch.stack((p[:, 1], p[:, 0] + each // 2), 1))
    assert torch.equal(r.ids.long(), route64(x, top_k, "softmax", bias)[0])


@pytest.mark.parametrize("experts,top_k", [(64, 33), (64, 64), (100, 50), (256, 40), (512, 64)])
def test_neighbouring_logits(experts, top_k):
    """More experts than the short list holds, whose fp32 logits are steps apart:
    in their order, without and with groups."""
    gen = torch.Generator(device=GPU)
    gen.manual_seed(1)
    x = 1 + torch.rand(200, experts, generator=gen, device=GPU).argsort(1).float() * 2.0 ** -23
    r = qw.route_experts(x, top_k)
    assert torch.equal(r.ids.long(), route64(x, top_k, "softmax", None)[0])
    if top_k <= experts // 2:
        r = qw.route_experts(-x, top_k, "sigmoid", groups=2, top_groups=1)
        assert torch.equal(r.ids.long(), route64(-x, top_k, "sigmoid", None, 2, 1)[0])


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("experts,scoring,groups,top_groups", [(256, "sigmoid", 8, 4), (256, "softmax", 1, 1), (64, "softmax", 1, 1),
                                                               (256, "softmax", 8, 4), (160, "sigmoid", 8, 3)])
def test_many_tokens(experts, scoring, groups, top_groups, seed):
    """16384 tokens, of which some have two groups or experts this close."""
    print("many", experts, scoring, groups, seed, flush=True)
    gen = torch.Generator(device=GPU)
    gen.manual_seed(100 + seed)
    popular = 0.7 * torch.randn(experts, generator=gen, device=GPU)
    x = 1.5 * torch.randn(16384, experts, generator=gen, device=GPU) + popular
    bias = -0.05 * popular
    r = qw.route_experts(x, 8, scoring, bias=bias, groups=groups, top_groups=top_groups)
    ids, w = route64(x, 8, scoring, bias, groups, top_groups)
    bad = (r.ids.long() != ids).any(1)
    assert not bad.any(), "tokens %s" % bad.nonzero()[:, 0].tolist()
    # fp64 to fp32: half a step of 2^-24; both sides' fp64 errors are far below it
    assert ((r.weights.double() - w).abs() <= 1.01 * 2.0 ** -24 * w).all()
    flat = r.ids.view(-1).long()
    rows = torch.sort(flat, stable=True).indices
    assert torch.equal(r.rows.long(), rows)
    assert torch.equal(r.offsets.long(), torch.nn.functional.pad(torch.bincount(flat, minlength=experts).cumsum(0), (1, 0)))
    assert torch.equal(r.places.view(-1)[rows].long(), torch.arange(len(rows), device=GPU))
