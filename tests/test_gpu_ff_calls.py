"""The feed-forward calls as a program makes them: captured and replayed, on
several streams and from several threads, behind padding; and what they refuse
on the GPU."""

import threading

import pytest

torch = pytest.importorskip("torch")
from test_gpu_kv_refusals import refuses  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16, BF16, I8, I32, F32 = torch.float16, torch.bfloat16, torch.int8, torch.int32, torch.float32
GPU = "cuda:0"


def say(*what):
    print(*what, flush=True)


def gen(seed):
    g = torch.Generator(device=GPU)
    g.manual_seed(seed)
    return g


def weight(seed, *shape):
    q = torch.randint(-127, 128, shape, dtype=I8, device=GPU, generator=gen(seed))
    s = ((torch.rand(shape[:-1], device=GPU, generator=gen(seed + 1)) + 0.5) * shape[-1] ** -0.5 / 64).half()
    return q, s


class Dense:
    """norm, gated product, product with the residual."""

    def __init__(self, tokens, hidden, inner, a8, dtype=F16):
        self.x = torch.zeros(tokens, hidden, dtype=dtype, device=GPU)
        self.h = torch.zeros_like(self.x)
        self.norm = (torch.rand(hidden, device=GPU, generator=gen(5)) + 0.5).to(dtype)
        self.up, self.down, self.a8, self.dtype = weight(1, 2 * inner, hidden), weight(3, hidden, inner), a8, dtype

    def __call__(self):
        if self.a8:
            q, s, h = qw.add_rms_norm(self.x, self.norm, residual=self.h, quantize=True)
            g = qw.w8a8_linear(q, s, *self.up, activation="silu", gated=True)
            return qw.w8a8_linear(*qw.quantize_activations(g), *self.down, residual=h, dtype=self.dtype)
        y, h = qw.add_rms_norm(self.x, self.norm, residual=self.h)
        return qw.w8a16_linear(qw.w8a16_linear(y, *self.up, activation="silu", gated=True), *self.down, residual=h)

    def feed(self, seed):
        self.x.copy_(torch.randn(self.x.shape, device=GPU, generator=gen(seed)))
        self.h.copy_(torch.randn(self.x.shape, device=GPU, generator=gen(seed + 1)))


class Sparse(Dense):
    """norm, router, experts, their sum."""

    def __init__(self, tokens, hidden, inner, experts, top_k, groups=1):
        super().__init__(tokens, hidden, inner, False)
        self.router = torch.randn(hidden, experts, device=GPU, generator=gen(7)).half() * hidden ** -0.5
        self.bias = torch.randn(experts, device=GPU, generator=gen(8)) * 0.05
        self.up, self.down = weight(1, experts, 2 * inner, hidden), weight(3, experts, hidden, inner)
        self.top_k, self.groups = top_k, groups

    def __call__(self):
        y, h = qw.add_rms_norm(self.x, self.norm, residual=self.h)
        route = qw.route_experts(y @ self.router, self.top_k, "sigmoid", self.bias, self.groups, max(1, self.groups // 2))
        g = qw.w8a16_experts(y, *self.up, route, activation="silu", gated=True)
        return qw.experts_combine(qw.w8a16_experts(g, *self.down, route, gather=False), route, residual=h)


STEPS = {
    "one token": lambda: Dense(1, 512, 1024, False),
    "tokens": lambda: Dense(40, 512, 1024, False),
    "few rows' parts": lambda: Dense(16, 512, 8192, False),
    "split": lambda: Dense(256, 512, 8192, False),
    "codes": lambda: Dense(40, 512, 1024, True),
    "split codes": lambda: Dense(250, 512, 8192, True),
    "one token's experts": lambda: Sparse(1, 512, 256, 16, 4),
    "experts": lambda: Sparse(50, 512, 256, 16, 4, groups=4),
    "many tokens' experts": lambda: Sparse(300, 512, 256, 8, 2),
}


def test_the_splits_are_reached():
    lib = qw.library()
    assert lib.qw_w8a16_linear_workspace(16, 512, 8192, 0) > 0
    assert lib.qw_w8a16_linear_workspace(256, 512, 8192, 0) > 0 and lib.qw_w8a8_linear_workspace(250, 512, 8192, 0) > 0


@pytest.mark.parametrize("name", STEPS)
def test_replayed(name):
    """A captured step, replayed over other inputs with eager work between,
    against the eager steps."""
    step = STEPS[name]()
    eager = []
    for seed in range(3):
        step.feed(10 * seed)
        eager.append(step())
    torch.cuda.synchronize()
    assert not torch.equal(eager[0], eager[1]) and all(torch.isfinite(e).all() for e in eager)
    say("capturing", name)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for again in range(3):
        for seed in range(3):
            step.feed(10 * seed)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager[seed])
            (step.x.float() * 2).sum().item()
            assert torch.equal(step(), eager[seed])


@pytest.mark.parametrize("first,second", [("split", "split codes"), ("experts", "many tokens' experts"),
                                          ("few rows' parts", "split")])
def test_two_graphs_of_one_pool(first, second):
    """Graphs that share their memory, and so their workspaces, replayed in
    turn on one stream."""
    steps, graphs, outs, pool = [STEPS[first](), STEPS[second]()], [], [], torch.cuda.graph_pool_handle()
    want = []
    for i, step in enumerate(steps):
        step.feed(i)
        want.append(step())
    for step in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = step()
        graphs.append(graph)
        outs.append(out)
    for again in range(4):
        for graph, out, w in zip(graphs, outs, want):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)


@pytest.mark.parametrize("a,b", [("split", "split codes"), ("experts", "many tokens' experts"), ("tokens", "one token's experts"),
                                 ("few rows' parts", "split codes")])
def test_two_streams(a, b):
    """Steps side by side on two streams, each with its own workspaces."""
    steps = [STEPS[a](), STEPS[b]()]
    for i, step in enumerate(steps):
        step.feed(i)
    want = [step() for step in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    for again in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(steps[i]())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_two_threads():
    steps = [STEPS["split"](), STEPS["experts"]()]
    for i, step in enumerate(steps):
        step.feed(i)
    want = [step() for step in steps]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [steps[i]() for _ in range(10)]
                torch.cuda.current_stream().synchronize()
                bad.extend(i for g in got if not torch.equal(g, want[i]))
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad, bad


def test_padding_rows_change_nothing():
    """A batch behind which rows of padding stand: NaN in the residual stream,
    -inf in the router's logits.  The tokens' rows are those of a batch without
    them as far as the kernels are the same (the skinny one here), and padding
    reaches no expert."""
    step = Sparse(12, 512, 256, 16, 4)
    step.feed(3)
    y, h = qw.add_rms_norm(step.x, step.norm, residual=step.h)
    logits = y @ step.router

    def rest(y, h, logits):
        route = qw.route_experts(logits, 4)
        g = qw.w8a16_experts(y, *step.up, route, activation="silu", gated=True)
        return route, qw.experts_combine(qw.w8a16_experts(g, *step.down, route, gather=False), route, residual=h)

    route, want = rest(y, h, logits)
    pad = lambda t, v: torch.cat((t, torch.full((5, t.shape[1]), v, dtype=t.dtype, device=GPU)))  # noqa: E731
    y2, h2 = qw.add_rms_norm(pad(step.x, float("nan")), step.norm, residual=pad(step.h, 1.0))
    assert torch.equal(y2[:12], y) and torch.equal(h2[:12], h) and y2[12:].isnan().all()
    route2, got = rest(y2, h2, pad(logits, -float("inf")))
    assert (route2.ids[12:] == -1).all() and route2.offsets[-1] == 48 and torch.equal(route2.ids[:12], route.ids)
    assert torch.equal(got[:12], want)
    assert got[12:].isnan().all()  # their own residual
    _, got = rest(y2, pad(h, 2.0), pad(logits, -float("inf")))
    assert (got[12:] == 2.0).all()


def t(shape, dtype=F16, device=GPU):
    return torch.zeros(shape, dtype=dtype, device=device)


def test_norm_refuses():
    good = dict(x=t((5, 64)), weight=t(64), residual=t((5, 64)))
    bad = [("x", None), ("x", lambda: t((5, 64), device="cpu")), ("x", lambda: t((5, 64), F32)), ("x", lambda: t((64, 5)).t()),
           ("x", lambda: t((5, 68))[:, :64]), ("x", lambda: t((1, 64)).expand(5, 64)), ("x", lambda: t((5, 65))[:, 1:]),
           ("x", lambda: t(320)), ("x", lambda: t((5, 64), BF16)), ("weight", lambda: t(63)), ("weight", lambda: t(128)[::2]),
           ("weight", None), ("residual", lambda: t((4, 64))), ("residual", lambda: t((5, 64), BF16)), ("residual", lambda: t((1, 64))),
           ("residual", lambda: t((5, 64), device="cpu")), ("eps", -1.0), ("eps", float("nan")), ("out", lambda: (t((5, 64)),)),
           ("out", lambda: (t((5, 60)), None)), ("out", lambda: t((5, 64)))]
    refuses(qw.add_rms_norm, good, bad, ())
    refuses(lambda **a: qw.add_rms_norm(**a, quantize=True), good, bad + [("out", lambda: (t((5, 64)), t(5), None))], ())
    with pytest.raises(qw.QwError):
        qw.add_rms_norm(t((2, 24)), t(24))
    x, w = t((5, 64)), t(64)
    for out in ((x, None), (t((5, 64)), x.view(-1)[:-8].as_strided((5, 56), (64, 1))), (w.expand(5, 64), None)):
        with pytest.raises((ValueError, TypeError, qw.QwError)):
            qw.add_rms_norm(x, w, residual=t((5, 64)), out=out)


LINEAR_BAD = [("q", lambda: t((32, 48), I8)), ("q", lambda: t((32, 64))), ("q", lambda: t((64, 32), I8).t()), ("q", None),
              ("q", lambda: t((32, 64), I8, "cpu")), ("scales", lambda: t(31)), ("scales", lambda: t(32, F32)), ("scales", lambda: t(64)[::2]),
              ("bias", lambda: t(31)), ("bias", lambda: t(32, F32)), ("bias", lambda: t(32, device="cpu")), ("residual", lambda: t((5, 31))),
              ("residual", lambda: t((1, 32)).expand(5, 32)), ("residual", lambda: t((5, 32), F32)), ("activation", "tanh"), ("activation", 1),
              ("gated", True), ("out", lambda: t((5, 33))), ("out", lambda: t((5, 32), F32)), ("out", lambda: t((5, 64))[:, ::2])]


def test_linear_refuses():
    good = dict(x=t((5, 64)), q=t((32, 64), I8), scales=t(32), bias=t(32), residual=t((5, 32)))
    refuses(qw.w8a16_linear, good, LINEAR_BAD + [
        ("x", lambda: t((5, 64), BF16)), ("x", lambda: t((5, 64), I8)), ("x", lambda: t((64, 5)).t()), ("x", lambda: t((5, 64), device="cpu")),
        ("x", None), ("x", lambda: t(64)), ("bias", lambda: t(32, BF16)), ("residual", lambda: t((5, 32), BF16))], ())
    with pytest.raises(ValueError):
        qw.w8a16_linear(t((5, 64)), t((31, 64), I8), t(31), gated=True)
    with pytest.raises(qw.QwError):
        qw.w8a16_linear(t((5, 24)), t((32, 24), I8), t(32))
    x = t((32, 64))
    with pytest.raises(qw.QwError):
        qw.w8a16_linear(x, t((64, 64), I8), t(64), out=x)


def test_w8a8_linear_refuses():
    for dtype in (F16, BF16):
        good = dict(qx=t((5, 64), I8), sx=t(5), q=t((32, 64), I8), scales=t(32), bias=t(32, dtype), residual=t((5, 32), dtype))
        other = BF16 if dtype is F16 else F16
        refuses(qw.w8a8_linear, good, LINEAR_BAD + [
            ("qx", lambda: t((5, 64))), ("qx", lambda: t((5, 48), I8)), ("qx", None), ("sx", None), ("sx", lambda: t(4)), ("sx", lambda: t(5, F32)),
            ("sx", lambda: t(10)[::2]), ("bias", lambda: t(32, other)), ("dtype", F32), ("dtype", other), ("out", lambda: t((5, 32), other))], ())


def test_route_refuses():
    good = dict(logits=t((9, 24)), top_k=3, bias=t(24, F32), groups=4, top_groups=2)
    refuses(qw.route_experts, good, [
        ("logits", None), ("logits", lambda: t((9, 24), I32)), ("logits", lambda: t((24, 9)).t()), ("logits", lambda: t((9, 48))[:, ::2]),
        ("logits", lambda: t((9, 24), device="cpu")), ("logits", lambda: t(24)), ("logits", lambda: t((9, 28))), ("logits", lambda: t((9, 520))),
        ("top_k", 0), ("top_k", 65), ("top_k", None), ("bias", lambda: t(24)), ("bias", lambda: t(23, F32)), ("bias", lambda: t(24, F32, "cpu")),
        ("groups", 5), ("groups", 0), ("groups", -1), ("top_groups", 5), ("top_groups", 0), ("scoring", "tanh"), ("scoring", None),
        ("scale", float("nan")), ("scale", float("inf"))], ())


def test_experts_refuse():
    route = qw.route_experts(torch.randn(6, 5, device=GPU, generator=gen(1)), 2)
    good = dict(x=t((6, 64)), q=t((5, 32, 64), I8), scales=t((5, 32)), route=route, bias=t((5, 32)))
    part = lambda **c: lambda: route._replace(**{k: v() for k, v in c.items()})  # noqa: E731
    refuses(qw.w8a16_experts, good, [
        ("x", None), ("x", lambda: t((12, 64))), ("x", lambda: t((6, 64), BF16)), ("x", lambda: t((64, 6)).t()), ("x", lambda: t((6, 48))),
        ("q", lambda: t((32, 64), I8)), ("q", lambda: t((4, 32, 64), I8)), ("q", lambda: t((5, 32, 64))), ("scales", lambda: t((5, 31))),
        ("scales", lambda: t(32)), ("bias", lambda: t(32)), ("bias", lambda: t((5, 32), F32)), ("route", None), ("route", lambda: tuple(route)),
        ("route", part(ids=lambda: t((6, 3), I32))), ("route", part(offsets=lambda: t(5, I32))), ("route", part(offsets=lambda: t(6, F32))),
        ("route", part(rows=lambda: t(11, I32))), ("route", part(rows=lambda: t(12, torch.int64))), ("route", part(rows=lambda: t(12, I32, "cpu"))),
        ("activation", "tanh"), ("gather", False), ("out", lambda: t((12, 16))), ("out", lambda: t((12, 32), F32))], ())
    with pytest.raises(qw.QwError):
        qw.w8a16_experts(t((6, 24)), t((5, 32, 24), I8), t((5, 32)), route)
    good = dict(y=t((12, 32)), route=route, residual=t((6, 32)))
    refuses(qw.experts_combine, good, [
        ("y", None), ("y", lambda: t((11, 32))), ("y", lambda: t((12, 32), BF16)), ("y", lambda: t((32, 12)).t()), ("route", None),
        ("route", part(places=lambda: t((6, 1), I32))), ("route", part(weights=lambda: t((6, 2)))), ("route", part(places=lambda: t((6, 2), F32))),
        ("residual", lambda: t((5, 32))), ("residual", lambda: t((6, 32), BF16)), ("residual", lambda: t((1, 32)).expand(6, 32)),
        ("out", lambda: t((6, 31))), ("out", lambda: t((6, 32), BF16))], ())
    y = t((12, 32))
    with pytest.raises(qw.QwError):
        qw.experts_combine(y, route, out=y[:6])
