"""The feed-forward half of a decoder layer with int8 weights, case by case: the residual's addition and RMS norm with an
output in 8 bits, the W8A16 and W8A8 products with bias, activation, gate and residual in their epilogue, the routing of
tokens to experts, and the experts' products with the sum over a token's experts.

``own`` false: each operator in elementary torch operations, in fp32 (the router's scores, which decide between experts, in
64 bits), rounded once.  ``own`` true: the calls a user makes of ``int8_weight_quantized_amd``.  ``exact`` gives the same
outputs from the definitions in 64 bits.

A weight is its int8 code times the fp16 scale of its output channel.  A gated product's weight holds the gate's channels
and then the other factor's.  A route lists its entries (a token and one of its experts) expert by expert: ``rows`` holds the
flat index token * top_k + place of each, ``offsets`` the first entry of each expert, ``places`` where each flat index went.
"""

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    """4096 channels with products of 4608 and 27392 is the layer of the benchmark's decode and prefill workloads (27392 is
    gate and up, 13696 each); 1024 to 4096 its encoder layer; experts of 2048 by 1024 are a generic layer of 64."""
    return [
        # one decode step of eight requests in front of an int8 product: launch latency
        norm_case("norm_decode", tokens=8, k=4096, dtype="f16", codes=True, residual=True),
        # ragged prompts of a wide bf16 model, in front of a 16-bit product
        norm_case("norm_wide", tokens=1021, k=8192, dtype="bf16", codes=False, residual=True),
        # a prompt batch in front of an int8 product
        norm_case("norm_prompt", tokens=16384, k=4096, dtype="f16", codes=True, residual=True),
        # one token's fused QKV projection with its bias
        linear_case("qkv_decode", m=1, n=4608, k=4096, bias=True),
        # gate and up of sixteen requests that decode
        linear_case("gate_up_decode", m=16, n=27392, k=4096, act="silu", gated=True),
        # gate and up of a prompt
        linear_case("gate_up_prompt", m=1024, n=27392, k=4096, act="silu", gated=True),
        # the down projection of ragged prompts, int8 activations, onto a bf16 residual stream
        linear_case("down_prompt_w8a8", m=2039, n=4096, k=13696, a8=True, dtype="bf16", residual=True),
        # a decode batch with an empty place: latency
        route_case("route_decode", tokens=64, experts=64, top=8, dtype="f16"),
        # a prompt batch with balanced, grouped experts
        route_case("route_prompt", tokens=16384, experts=256, top=8, dtype="f32", sigmoid=True, bias=True, groups=8, top_groups=4),
        # gate and up of a decode batch: most experts have a few rows
        experts_case("experts_up_decode", tokens=32, experts=64, top=8, n=2048, k=2048, gated=True),
        # down and the sum over experts of the same batch
        experts_case("experts_down_decode", tokens=32, experts=64, top=8, n=2048, k=1024, down=True),
        # gate and up of ragged prompts
        experts_case("experts_up_prompt", tokens=4099, experts=64, top=6, n=2048, k=2048, gated=True),
    ]


def norm_case(name, tokens, k, dtype, codes, residual):
    return named(name, {"op": "norm", "tokens": tokens, "k": k, "dtype": dtype, "codes": codes, "residual": residual})


def linear_case(name, m, n, k, a8=False, dtype="f16", bias=False, act="none", gated=False, residual=False):
    return named(name, {"op": "linear", "m": m, "n": n, "k": k, "a8": a8, "dtype": dtype, "bias": bias, "act": act, "gated": gated,
                        "residual": residual})


def route_case(name, tokens, experts, top, dtype, sigmoid=False, bias=False, groups=1, top_groups=1, renormalize=True):
    return named(name, {"op": "route", "tokens": tokens, "experts": experts, "top": top, "dtype": dtype, "sigmoid": sigmoid,
                        "bias": bias, "groups": groups, "top_groups": top_groups, "renormalize": renormalize})


def experts_case(name, tokens, experts, top, n, k, gated=False, down=False, bias=False):
    return named(name, {"op": "experts", "tokens": tokens, "experts": experts, "top": top, "n": n, "k": k, "gated": gated,
                        "down": down, "bias": bias})


def named(name, case):
    return dict({"name": name}, **case) if name else case


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    def coin():
        return rng.random() < 0.5

    op = rng.choice(("norm", "linear", "linear", "route", "experts", "experts"))
    if op == "norm":
        k = 16 * log(16, 1024)
        return norm_case(None, log(1, min(16384, 16384 * 4096 // k)), k, rng.choice(("f16", "bf16")), coin(), rng.random() < 0.8)
    if op == "linear":
        a8, gated = coin(), coin()
        k = 16 * log(16, 856)
        n = log(256, 27392)
        n += n % 2 if gated else 0
        m = log(1, min(2048, 100_000_000_000 // (n * k)))
        return linear_case(None, m, n, k, a8, rng.choice(("f16", "bf16")) if a8 else "f16", coin(),
                           rng.choice(("silu", "gelu", "gelu_tanh")) if gated else rng.choice(("none", "none", "relu", "gelu", "silu")),
                           gated, coin() and not gated)
    if op == "route":
        experts, groups, top_groups = rng.choice(((8, 1, 1), (16, 1, 1), (60, 1, 1), (64, 1, 1), (128, 1, 1), (160, 8, 3), (256, 8, 4)))
        sigmoid = coin()
        return route_case(None, log(1, 16384), experts, rng.choice((1, 2, 4, 6, 8)), rng.choice(("f16", "bf16", "f32")), sigmoid,
                          sigmoid and coin(), groups, top_groups, rng.random() < 0.8)
    experts = rng.choice((8, 16, 32, 60, 64, 128))
    top = rng.choice((1, 2, 4, 6, 8))
    k, n = 16 * log(16, 256), log(256, 4096)
    gated = coin()
    n += n % 2 if gated else 0
    while experts * n * k > 1 << 29:
        k = max(256, k // 2 // 16 * 16)
        n = max(256, n // 2 // 2 * 2)
    tokens = log(1, min(4096, 100_000_000_000 // (top * n * k)))
    return experts_case(None, tokens, experts, top, n, k, gated, not gated, coin())


def work(case):
    if case["op"] == "norm":
        T, k = case["tokens"], case["k"]
        row = k * (2.0 + (4.0 if case["residual"] else 0.0) + (1.0 if case["codes"] else 2.0))
        return {"bytes": T * (row + (2.0 if case["codes"] else 0.0)) + 2.0 * k, "flops": 6.0 * T * k}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        out = n // 2 if case["gated"] else n
        b = n * (k + 2.0) + m * k * (1.0 if case["a8"] else 2.0) + (2.0 * m if case["a8"] else 0.0) + 2.0 * m * out
        return {"bytes": b + (2.0 * n if case["bias"] else 0.0) + (2.0 * m * out if case["residual"] else 0.0), "flops": 2.0 * m * n * k}
    T, E, top = case["tokens"], case["experts"], case["top"]
    if case["op"] == "route":
        return {"bytes": T * (E * (4.0 if case["dtype"] == "f32" else 2.0) + 16.0 * top) + 4.0 * (E + 1), "flops": 10.0 * T * E}
    n, k = case["n"], case["k"]
    entries, hit = T * top, E * (1.0 - (1.0 - top / E) ** T)  # the weights of the experts that have a token
    b = hit * n * (k + 2.0 + (2.0 if case["bias"] else 0.0)) + 4.0 * entries
    if case["down"]:  # every entry's row in; the residual in and the sum out
        b += 2.0 * entries * k + 8.0 * entries + 4.0 * T * n
    else:  # every token's row in; every entry's row out
        b += 2.0 * T * k + 2.0 * entries * (n // 2 if case["gated"] else n)
    return {"bytes": b, "flops": 2.0 * entries * n * k}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def weight(gen, *shape):
    """int8 codes and fp16 scales of a normal weight whose product keeps the size of its input."""
    codes = normal(gen, *shape).mul_(127 / 3.5).round_().clamp_(-127, 127).to(torch.int8)
    spread = 0.7 + 0.6 * torch.rand(*shape[:-1], generator=gen, device=DEV)
    return codes, (spread * (3.5 / 127 / math.sqrt(shape[-1]))).half()


def stream(gen, tokens, k):
    """A residual stream: a few channels are much larger than the rest."""
    gain = torch.ones(k, device=DEV)
    gain[torch.randint(0, k, (4,), generator=gen, device=DEV)] = 20.0
    return normal(gen, tokens, k) * gain


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, k, dtype = case["tokens"], case["k"], TYPES[case["dtype"]]
        s["x"] = normal(gen, T, k).to(dtype)
        s["res"] = stream(gen, T, k).to(dtype) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * normal(gen, k)).to(dtype)
        return s
    if case["op"] == "linear":
        m, n, k, dtype = case["m"], case["n"], case["k"], TYPES[case["dtype"]]
        s["q"], s["scales"] = weight(gen, n, k)
        if case["a8"]:
            s["x"], s["sx"] = weight(gen, m, k)
            s["sx"] = (s["sx"].float() * math.sqrt(k)).half()
        else:
            s["x"] = normal(gen, m, k).half()
        s["b"] = (0.2 * normal(gen, n)).to(dtype) if case["bias"] else None
        s["res"] = stream(gen, m, n // 2 if case["gated"] else n).to(dtype) if case["residual"] else None
        return s
    T, E, top = case["tokens"], case["experts"], case["top"]
    popular = 0.7 * normal(gen, E)  # some experts are asked for more often
    if case["op"] == "route":
        logits = 1.5 * normal(gen, T, E) + popular
        if T >= 8:
            logits[-1] = -math.inf  # a batch's empty place goes to no expert
        s["logits"] = logits.to(TYPES[case["dtype"]])
        s["bias_e"] = -0.05 * popular if case["bias"] else None
        return s
    ids = (1.5 * normal(gen, T, E) + popular).topk(top, dim=1).indices.to(torch.int32)
    w = torch.rand(T, top, generator=gen, device=DEV) + 0.1
    w = w / w.sum(1, keepdim=True)
    if T >= 8:
        ids[-1], w[-1] = -1, 0.0
    s["ids"], s["w"] = ids, w
    s["offsets"], s["rows"], s["places"] = listing(ids, E)
    s["used"] = int(s["offsets"][-1])
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    s["q"], s["scales"] = weight(gen, E, case["n"], case["k"])
    s["b"] = (0.2 * normal(gen, E, case["n"])).half() if case["bias"] else None
    s["x"] = normal(gen, T * top if case["down"] else T, case["k"]).half()
    s["res"] = stream(gen, T, case["n"]).half() if case["down"] else None
    return s


def listing(ids, experts):
    """offsets, rows and places of a route: its entries expert by expert, in their order."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.nn.functional.pad(torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0), (1, 0))
    at = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(at < offsets[-1], order, -1)
    places = torch.empty_like(order)
    places[order] = at
    places = torch.where(flat < 0, -1, places)
    return offsets.to(torch.int32), rows.to(torch.int32), places.view(ids.shape).to(torch.int32)


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def values(codes, scales, dtype):
    """What int8 codes with a scale a row stand for."""
    return (codes.float() * scales.float()[:, None]).to(dtype)


def own_norm(s):
    import int8_weight_quantized_amd as qw
    if s["codes"]:
        q, scales, h = qw.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS, quantize=True)
        y = values(q, scales, s["x"].dtype)
    else:
        y, h = qw.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS)
    return {"y": y, "h": h}


def own_linear(s):
    import int8_weight_quantized_amd as qw
    more = {"bias": s["b"], "activation": None if s["act"] == "none" else s["act"], "gated": s["gated"], "residual": s["res"]}
    if s["a8"]:
        return {"y": qw.w8a8_linear(s["x"], s["sx"], s["q"], s["scales"], dtype=TYPES[s["dtype"]], **more)}
    return {"y": qw.w8a16_linear(s["x"], s["q"], s["scales"], **more)}


def own_route(s):
    import int8_weight_quantized_amd as qw
    r = qw.route_experts(s["logits"], s["top"], scoring="sigmoid" if s["sigmoid"] else "softmax", bias=s["bias_e"],
                         groups=s["groups"], top_groups=s["top_groups"], renormalize=s["renormalize"])
    return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "places": r.places}


def own_experts(s):
    import int8_weight_quantized_amd as qw
    route = qw.ExpertRoute(s["ids"], s["w"], s["offsets"], s["rows"], s["places"])
    if s["down"]:
        y = qw.w8a16_experts(s["x"], s["q"], s["scales"], route, bias=s["b"], gather=False, dtype=torch.float32)
        return {"out": qw.experts_combine(y, route, residual=s["res"])}
    return {"y": qw.w8a16_experts(s["x"], s["q"], s["scales"], route, bias=s["b"], activation="silu" if s["gated"] else None,
                                  gated=s["gated"])}


def plain_norm(s):
    x = s["x"].float()
    h = s["x"] if s["res"] is None else (x + s["res"].float()).to(s["x"].dtype)
    x = h.float()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if not s["codes"]:
        return {"y": y.to(h.dtype), "h": h}
    scales = (y.abs().amax(1) / 127.0).half()
    codes = torch.round(y / scales.float()[:, None]).clamp(-127, 127).nan_to_num(0.0).to(torch.int8)
    return {"y": values(codes, scales, h.dtype), "h": h}


def activate(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def plain_linear(s):
    w = s["q"].float() * s["scales"].float()[:, None]
    x = s["x"].float() * s["sx"].float()[:, None] if s["a8"] else s["x"].float()
    y = x @ w.t()
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = activate(gate, s["act"]) * up
    else:
        y = activate(y, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(TYPES[s["dtype"]])}


def plain_route(s):
    x = s["logits"].double()
    live = x > -math.inf
    if s["sigmoid"]:
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    p = torch.where(live, p, 0.0)
    c = x if s["bias_e"] is None else torch.where(live, p + s["bias_e"].double(), -math.inf)
    T, E = c.shape
    if s["groups"] > 1:
        by = c.view(T, s["groups"], -1)
        score = by.amax(2) if s["bias_e"] is None else by.topk(2, dim=2).values.sum(2)
        first = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, first, True)
        c = torch.where(keep[:, :, None], by, -math.inf).view(T, E)
    best = torch.sort(c, dim=1, descending=True, stable=True)
    ids = best.indices[:, :s["top"]]
    found = best.values[:, :s["top"]] > -math.inf
    w = torch.where(found, p.gather(1, ids), 0.0)
    if s["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    ids = torch.where(found, ids, -1).to(torch.int32)
    offsets, rows, places = listing(ids, E)
    return {"ids": ids, "weights": w.float(), "offsets": offsets, "rows": rows, "places": places}


def plain_experts(s):
    E, used, most = s["experts"], s["used"], s["most"]
    offsets, rows = s["offsets"].long(), s["rows"][:used].long()
    at = torch.arange(used, device=rows.device)
    e = torch.searchsorted(offsets[1:], at, right=True)
    slot = e * most + at - offsets[e]  # each expert's rows, padded to the most that one has
    x = torch.zeros(E * most, s["k"], device=rows.device)
    x[slot] = (s["x"][:used] if s["down"] else s["x"][rows // s["top"]]).float()
    w = s["q"].float() * s["scales"].float()[:, :, None]
    y = torch.bmm(w, x.view(E, most, -1).transpose(1, 2).contiguous())
    y = y.transpose(1, 2).reshape(E * most, -1)[slot]
    if s["b"] is not None:
        y = y + s["b"].float()[e]
    if s["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = activate(gate, "silu") * up
    whole = torch.zeros(s["rows"].numel(), y.shape[1], device=y.device)  # entries of no expert are zero
    whole[:used] = y
    if not s["down"]:
        return {"y": whole.half()}
    each = whole[s["places"].clamp(min=0).long()] * s["w"][:, :, None]  # (a weight of 0 where a place is empty)
    return {"out": (s["res"].float() + each.sum(1)).half()}


OWN = {"norm": own_norm, "linear": own_linear, "route": own_route, "experts": own_experts}
PLAIN = {"norm": plain_norm, "linear": plain_linear, "route": plain_route, "experts": plain_experts}


# ---------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    return {"norm": exact_norm, "linear": exact_linear, "route": exact_route, "experts": exact_experts}[case["op"]](prepare(case, seed))


def exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = (h + s["res"].double()).to(s["x"].dtype).double()
    y = s["weight"].double() * h * (h.square().sum(1) / h.shape[1] + EPS).rsqrt()[:, None]
    if s["codes"]:
        step = (y.abs().amax(1) / 127.0).half().double()[:, None]
        y = torch.where(step > 0, (y / step).round().clamp(-127, 127) * step, 0.0)
    return {"y": y, "h": h}


def act64(x, act):
    if act == "relu":
        return x.clamp(min=0.0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def product64(x, q, scales, bias, act, gated):
    y = (x @ q.double().t()) * scales.double()
    if bias is not None:
        y += bias.double()
    half = y.shape[1] // 2
    return act64(y[:, :half], act) * y[:, half:] if gated else act64(y, act)


def exact_linear(s):
    x = s["x"].double()
    if s["a8"]:
        x = x * s["sx"].double()[:, None]
    y = product64(x, s["q"], s["scales"], s["b"], s["act"], s["gated"])
    return {"y": y if s["res"] is None else y + s["res"].double()}


def exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    p = torch.sigmoid(x) if s["sigmoid"] else torch.softmax(x, 1).nan_to_num(0.0)
    c = x if s["bias_e"] is None else (p + s["bias_e"]).masked_fill(torch.isinf(x), -math.inf)
    index = torch.arange(E, device=x.device)
    per = E // s["groups"]

    def best(c):
        """The largest of each row, and its lowest index."""
        top = c.amax(1, keepdim=True)
        return top[:, 0], torch.where(c == top, torch.arange(c.shape[1], device=c.device), c.shape[1]).amin(1)

    if s["groups"] > 1:
        score = []
        for g in range(s["groups"]):
            part = c[:, g * per:(g + 1) * per]
            first, at = best(part)
            score.append(first if s["bias_e"] is None else first + best(part.scatter(1, at[:, None], -math.inf))[0])
        score = torch.stack(score, 1)
        kept = torch.zeros(T, E, dtype=torch.bool, device=x.device)
        for _ in range(s["top_groups"]):
            _, at = best(score)
            kept |= index // per == at[:, None]
            score = score.scatter(1, at[:, None], -math.inf)
        c = c.masked_fill(~kept, -math.inf)
    w = []
    for _ in range(s["top"]):
        top, at = best(c)
        w.append(torch.where(top > -math.inf, p.gather(1, at[:, None])[:, 0], 0.0))
        c = c.scatter(1, at[:, None], -math.inf)
    w = torch.stack(w, 1)
    if s["renormalize"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return {"ids": None, "weights": w, "offsets": None, "rows": None, "places": None}


def exact_experts(s):
    offsets = s["offsets"].tolist()
    ids = s["ids"].reshape(-1)
    y = torch.zeros(ids.numel(), s["n"] // 2 if s["gated"] else s["n"], dtype=torch.float64, device=ids.device)
    for e in range(s["experts"]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        mine = torch.nonzero(ids == e)[:, 0]
        x = (s["x"][lo:hi] if s["down"] else s["x"][mine // s["top"]]).double()
        b = None if s["b"] is None else s["b"][e]
        y[lo:hi] = product64(x, s["q"][e], s["scales"][e], b, "silu" if s["gated"] else "none", s["gated"])
    if not s["down"]:
        return {"y": y}
    out = s["res"].double()
    for j in range(s["top"]):
        at = s["places"][:, j].long()
        out += torch.where(at[:, None] < 0, 0.0, s["w"][:, j].double()[:, None] * y[at.clamp(min=0)])
    return {"out": out}
