"""The feed-forward operators in 64 bits, from their definitions, for the tests:
plain torch in float64 (products) and plain Python (the router)."""

import math

import torch

# half a step of a rounding, relative to the value, and half the smallest step
HALF = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float32: (2.0 ** -24, 2.0 ** -150)}


def act64(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if act == "silu":
        return x * torch.sigmoid(x)
    return x


def linear64(x, q, scales, bias=None, act=None, gated=False, residual=None, sx=None):
    """(result, how far fp32 may be from it before the final rounding)."""
    v = (x.double() @ q.double().t()) * scales.double()
    if sx is not None:
        v = v * sx.double()[:, None]
    # the sums of these tests are exact in fp32 (integers below 2^24); scale and
    # bias are a product of two exact numbers and one fused add: 2^-23 of the
    # larger of both covers them
    off = 2.0 ** -23 * v.abs()
    if bias is not None:
        v = v + bias.double()
        off = off + 2.0 ** -23 * bias.double().abs()
    # an activation within 2^-17 of its result, or of v in the negative tails,
    # and v's own error, which no activation amplifies by more than 1.13
    def with_error(v, off):
        a = act64(v, act)
        tail = torch.where(v < -6, v.abs(), a.abs())
        return a, 1.13 * off + (2.0 ** -17 * tail if act not in (None, "relu") else 0)
    if gated:
        half = v.shape[1] // 2
        a, ea = with_error(v[:, :half], off[:, :half])
        b, eb = v[:, half:], off[:, half:]
        y, off = a * b, ea * b.abs() + eb * a.abs() + ea * eb + 2.0 ** -24 * (a * b).abs()
    else:
        y, off = with_error(v, off)
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -24 * y.abs()
    return y, off


def assert_rounded(got, want, off):
    """got is want within `off` and one rounding to its type.  A value beyond
    the type's largest is infinity."""
    rel, least = HALF[got.dtype]
    assert got.shape == want.shape
    g = got.double()
    top = torch.finfo(got.dtype).max
    inf = g.isinf()
    assert not (inf & (want.abs() * (1 + rel) + off < top)).any(), "infinite where the value fits"
    assert not g.isnan().any()
    bad = ~inf & ((g - want).abs() > off * (1 + rel) + rel * want.abs() + least)
    assert not bad.any(), "%d of %d off, worst %g of its bound, first at %s: %g for %g" % (
        bad.sum(), bad.numel(), ((g - want).abs() / (off * (1 + rel) + rel * want.abs() + least))[~inf].max(),
        bad.nonzero()[0].tolist(), g[bad][0], want[bad][0])


def integers(gen, shape, most, dtype, device="cuda"):
    return torch.randint(-most, most + 1, shape, generator=gen, device=device).to(dtype)


def scale16(gen, shape, size, device="cuda"):
    return ((0.5 + torch.rand(shape, generator=gen, device=device)) * size).half()


def route64(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """Lists: ids and weights of each token (plain Python over float64)."""
    ids, weights = [], []
    for row in logits.double().tolist():
        E = len(row)
        big = 3.4028234663852886e38
        l = [min(v, big) if v > -math.inf else -math.inf for v in row]  # (NaN compares false)
        live = [v > -math.inf for v in l]
        if scoring == "sigmoid":
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in l]
        else:
            m = max(l)
            e = [math.exp(v - m) if ok else 0.0 for v, ok in zip(l, live)]
            t = sum(e)
            s = [v / t if t else 0.0 for v in e]
        if bias is None:
            c = l
        else:
            c = [s[i] + b if live[i] else -math.inf for i, b in enumerate(bias.double().tolist())]
            c = [v if v > -math.inf else -math.inf for v in c]
        if groups > 1:
            size = E // groups
            score = []
            for g in range(groups):
                part = sorted((v for v in c[g * size:(g + 1) * size]), reverse=True)
                if bias is not None and size > 1 and part[1] > -math.inf:
                    score.append(part[0] + part[1])
                else:
                    score.append(part[0])
            first = sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups]
            kept = {g for g in first if score[g] > -math.inf}
            c = [v if i // size in kept else -math.inf for i, v in enumerate(c)]
        best = [i for i in sorted(range(E), key=lambda i: (-c[i], i)) if c[i] > -math.inf][:top_k]
        w = [s[i] for i in best]
        if renormalize:
            t = sum(w)
            w = [v / t if t > 0 else 0.0 for v in w]
        ids.append(best + [-1] * (top_k - len(best)))
        weights.append([v * scale for v in w] + [0.0] * (top_k - len(best)))
    return ids, weights


def listing(ids, experts):
    """offsets, rows and places of a route (lists)."""
    flat = [i for row in ids for i in row]
    by = [[f for f, e in enumerate(flat) if e == x] for x in range(experts)] if len(flat) < 4000 else None
    if by is None:
        by = [[] for _ in range(experts)]
        for f, e in enumerate(flat):
            if e >= 0:
                by[e].append(f)
    offsets, rows = [0], []
    for b in by:
        rows += b
        offsets.append(len(rows))
    places = [-1] * len(flat)
    for p, f in enumerate(rows):
        places[f] = p
    return offsets, rows + [-1] * (len(flat) - len(rows)), places


def made_route(ids, weights=None):
    """An ExpertRoute on the GPU from a list of rows of expert ids; `experts`
    is the caller's: offsets come from listing()."""
    import int8_weight_quantized_amd as qw

    def build(experts):
        offsets, rows, places = listing(ids, experts)
        i = torch.tensor(ids, dtype=torch.int32, device="cuda")
        w = torch.ones(i.shape, device="cuda") if weights is None else weights
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return qw.ExpertRoute(i, w, t(offsets), t(rows), t(places).view(i.shape))
    return build
