"""The feed-forward calls without a GPU: what the C ABI rejects, and what the
binding rejects before a pointer reaches it."""

import pytest

torch = pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")

META = torch.device("meta")
OK, INVALID, MISALIGNED, UNSUPPORTED, LAUNCH = (qw.QW_SUCCESS, qw.QW_ERROR_INVALID_VALUE, qw.QW_ERROR_MISALIGNED,
                                                qw.QW_ERROR_UNSUPPORTED, qw.QW_ERROR_LAUNCH)
NAN, INF = float("nan"), float("inf")

# never dereferenced: every call is rejected on the host, or has nothing to do
P = [(i + 1) << 40 for i in range(16)]


def call(name, args, **changes):
    args = dict(args)
    args.update(changes)
    return getattr(qw.library(), name)(*args.values())


NORM = dict(x=P[0], x_stride=64, res=P[1], res_stride=64, weight=P[2], dtype=0, tokens=5, k=64, eps=1e-6, h=P[3], h_stride=64, y=P[4],
            stream=None)
CODES = dict(x=P[0], x_stride=64, res=P[1], res_stride=64, weight=P[2], dtype=1, tokens=5, k=64, eps=1e-6, h=P[3], h_stride=64, q=P[4],
             scales=P[5], stream=None)
NORM_BAD = [
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(tokens=-1), INVALID), (dict(k=0), INVALID), (dict(k=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(x=0), INVALID), (dict(weight=0), INVALID),
    (dict(res=0), INVALID), (dict(h=0), INVALID), (dict(x_stride=56), INVALID), (dict(res_stride=56), INVALID), (dict(h_stride=0), INVALID),
    (dict(k=56, x_stride=64), UNSUPPORTED), (dict(k=65552, x_stride=65552, res_stride=65552, h_stride=65552), UNSUPPORTED),
    (dict(x_stride=68), UNSUPPORTED), (dict(res_stride=66), UNSUPPORTED), (dict(h_stride=(1 << 31) + 8), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(x=P[0] + 8), MISALIGNED), (dict(weight=P[2] + 2), MISALIGNED), (dict(h=P[3] + 4), MISALIGNED),
    (dict(h=P[0] + 16), INVALID), (dict(h=P[1] + 128), INVALID), (dict(h=P[2]), INVALID), (dict(h=P[4]), INVALID),
    (dict(h=P[0], h_stride=72), INVALID),                                                                    # in place, at another stride
    (dict(x=P[0], x_stride=128, h=P[0] + 64, h_stride=128), INVALID),                                        # columns that overlap
]


@pytest.mark.parametrize("changes,status", NORM_BAD + [(dict(y=0), INVALID), (dict(y=P[4] + 2), MISALIGNED), (dict(y=P[0]), INVALID),
                                                       (dict(y=P[1] + 512), INVALID), (dict(y=P[2]), INVALID)])
def test_norm_rejects(changes, status):
    assert call("qw_add_rms_norm", NORM, **changes) == status


@pytest.mark.parametrize("changes,status", NORM_BAD + [(dict(q=0), INVALID), (dict(scales=0), INVALID), (dict(q=P[4] + 1), MISALIGNED),
                                                       (dict(scales=P[5] + 2), MISALIGNED), (dict(scales=P[4] + 304), INVALID),
                                                       (dict(q=P[3]), INVALID), (dict(scales=P[2] + 112), INVALID)])
def test_norm_quantize_rejects(changes, status):
    assert call("qw_add_rms_norm_quantize", CODES, **changes) == status


LINEAR = dict(x=P[0], q=P[1], scales=P[2], bias=P[3], act=4, gated=0, res=P[4], y=P[5], m=40, n=64, k=128, path=0, tile=0, splits=1,
              ws=None, ws_bytes=0, stream=None)
A8 = dict(qx=P[0], sx=P[6], q=P[1], scales=P[2], bias=P[3], act=4, gated=0, res=P[4], dtype=1, y=P[5], m=40, n=64, k=128, path=0, tile=0,
          splits=1, ws=None, ws_bytes=0, stream=None)
LINEAR_BAD = [
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(gated=2), INVALID), (dict(gated=1, n=63), INVALID), (dict(m=-1), INVALID),
    (dict(n=-1), INVALID), (dict(k=0), INVALID), (dict(path=4), INVALID), (dict(path=-1), INVALID), (dict(tile=256256), INVALID),
    (dict(path=3, tile=256256), INVALID), (dict(path=2, tile=12), INVALID), (dict(path=2, tile=256128, splits=2), INVALID),
    (dict(path=2, tile=256256, splits=0), INVALID), (dict(path=2, tile=256256, splits=65), INVALID), (dict(splits=2), INVALID),
    (dict(path=2, tile=256256, splits=2), INVALID),                                                          # no workspace
    (dict(path=2, tile=256256, splits=2, ws=P[7], ws_bytes=2 * 262144 - 1), INVALID),
    (dict(path=2, tile=256256, splits=2, ws=P[5], ws_bytes=2 * 262144), INVALID),
    (dict(path=2, tile=256256, splits=2, ws=P[7] + 8, ws_bytes=2 * 262144), MISALIGNED),
    (dict(path=2, tile=256256, splits=3, ws=P[7], ws_bytes=1 << 23), UNSUPPORTED),                           # k < 64 splits
    (dict(ws_bytes=-1), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(q=0), INVALID), (dict(scales=0), INVALID), (dict(y=0), INVALID), (dict(k=120), UNSUPPORTED), (dict(m=1 << 31), UNSUPPORTED),
    (dict(n=1 << 31), UNSUPPORTED), (dict(q=P[1] + 8), MISALIGNED), (dict(bias=P[3] + 2), MISALIGNED), (dict(res=P[4] + 8), MISALIGNED),
    (dict(y=P[5] + 2), MISALIGNED), (dict(y=P[0] + 16), INVALID), (dict(y=P[1]), INVALID), (dict(y=P[2]), INVALID), (dict(y=P[3] + 112), INVALID),
    (dict(y=P[4] + 16), INVALID), (dict(res=P[5] + 16), INVALID),
]


@pytest.mark.parametrize("changes,status", LINEAR_BAD + [(dict(x=0), INVALID), (dict(path=1), UNSUPPORTED), (dict(path=1, m=3), UNSUPPORTED),
                                                         (dict(path=1, m=1, gated=1, k=8208), UNSUPPORTED),
                                                         (dict(path=2, k=1 << 24), UNSUPPORTED), (dict(x=P[0] + 4), MISALIGNED),
                                                         (dict(path=2, tile=256256, k=1 << 23, n=16, m=1), UNSUPPORTED),
                                                         (dict(path=2, gated=1, n=1 << 20, k=4096), UNSUPPORTED),
                                                         (dict(path=3, m=16 * 65535 + 1, n=2, k=16, bias=0, res=0), UNSUPPORTED)])
def test_linear_rejects(changes, status):
    assert call("qw_w8a16_linear_path", LINEAR, **changes) == status


@pytest.mark.parametrize("changes,status", LINEAR_BAD + [(dict(qx=0), INVALID), (dict(sx=0), INVALID), (dict(dtype=2), INVALID), (dict(path=1), INVALID),
                                                         (dict(path=2, tile=128128), INVALID), (dict(k=131088), UNSUPPORTED),
                                                         (dict(sx=P[6] + 2), MISALIGNED), (dict(y=P[6]), INVALID)])
def test_w8a8_linear_rejects(changes, status):
    assert call("qw_w8a8_linear_path", A8, **changes) == status


ROUTE = dict(logits=P[0], dtype=2, tokens=70, experts=30, top_k=4, scoring=1, bias=P[1], groups=3, top_groups=2, renorm=1, scale=1.0, ids=P[2],
             weights=P[3], offsets=P[4], rows=P[5], places=P[6], ws=P[7], ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dtype=3), INVALID), (dict(tokens=-1), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID), (dict(scoring=2), INVALID),
    (dict(groups=0), INVALID), (dict(groups=4), INVALID), (dict(top_groups=0), INVALID), (dict(top_groups=4), INVALID), (dict(renorm=2), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(logits=0), INVALID), (dict(ids=0), INVALID), (dict(weights=0), INVALID),
    (dict(offsets=0), INVALID), (dict(rows=0), INVALID), (dict(places=0), INVALID), (dict(ws=0), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(ws_bytes=-1), INVALID), (dict(experts=513, groups=1, top_groups=1), UNSUPPORTED), (dict(top_k=65), UNSUPPORTED),
    (dict(experts=130, groups=65), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED), (dict(logits=P[0] + 4), MISALIGNED),
    (dict(bias=P[1] + 8), MISALIGNED), (dict(ids=P[2] + 2), MISALIGNED), (dict(ws=P[7] + 4), MISALIGNED),
    (dict(ids=P[0] + 64), INVALID), (dict(rows=P[1]), INVALID), (dict(places=P[5] + 1116), INVALID), (dict(offsets=P[3] + 4), INVALID),
    (dict(ws=P[6]), INVALID),
])
def test_route_rejects(changes, status):
    assert call("qw_route_experts", ROUTE, **changes) == status


EXPERTS = dict(x=P[0], x_rows=20, gather=1, q=P[1], scales=P[2], bias=P[3], act=4, gated=1, offsets=P[4], rows=P[5], entries=40, top_k=2, y=P[6],
               experts=5, n=64, k=128, path=0, tile=0, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(act=9), INVALID), (dict(gated=2), INVALID), (dict(n=63), INVALID), (dict(x_rows=-1), INVALID), (dict(entries=-1), INVALID),
    (dict(gather=2), INVALID), (dict(gather=0), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID), (dict(k=0), INVALID),
    (dict(path=1), INVALID), (dict(tile=256128), INVALID), (dict(path=2, tile=128128), INVALID), (dict(path=3, tile=128064), INVALID),
    (dict(x=0), INVALID), (dict(q=0), INVALID), (dict(scales=0), INVALID), (dict(offsets=0), INVALID), (dict(rows=0), INVALID), (dict(y=0), INVALID),
    (dict(k=120), UNSUPPORTED), (dict(experts=513), UNSUPPORTED), (dict(entries=1 << 31), UNSUPPORTED), (dict(k=1 << 24), UNSUPPORTED),
    (dict(n=1 << 20, k=4096), UNSUPPORTED), (dict(x_rows=1 << 20, k=4096), UNSUPPORTED), (dict(path=3, entries=(1 << 19) + 1), UNSUPPORTED),
    (dict(path=2, tile=256256, k=1 << 23, n=2, x_rows=1), UNSUPPORTED),
    (dict(x=P[0] + 2), MISALIGNED), (dict(q=P[1] + 8), MISALIGNED), (dict(offsets=P[4] + 2), MISALIGNED), (dict(rows=P[5] + 1), MISALIGNED),
    (dict(y=P[0] + 256), INVALID), (dict(y=P[1] + 5 * 64 * 128 - 16), INVALID), (dict(y=P[2]), INVALID), (dict(y=P[3]), INVALID),
    (dict(y=P[4]), INVALID), (dict(y=P[5] + 144), INVALID),
])
def test_experts_rejects(changes, status):
    assert call("qw_w8a16_experts_path", EXPERTS, **changes) == status


COMBINE = dict(y=P[0], entries=40, places=P[1], weights=P[2], tokens=20, top_k=2, res=P[3], out=P[4], n=64, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(entries=-1), INVALID), (dict(tokens=-1), INVALID), (dict(top_k=0), INVALID), (dict(n=-1), INVALID), (dict(y=0), INVALID),
    (dict(places=0), INVALID), (dict(weights=0), INVALID), (dict(out=0), INVALID), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(entries=1 << 31), UNSUPPORTED), (dict(tokens=1 << 30, n=1 << 11), UNSUPPORTED), (dict(y=P[0] + 8), MISALIGNED),
    (dict(places=P[1] + 2), MISALIGNED), (dict(out=P[4] + 2), MISALIGNED), (dict(out=P[0]), INVALID), (dict(out=P[1] + 144), INVALID),
    (dict(out=P[2]), INVALID), (dict(out=P[3] + 16), INVALID),
])
def test_combine_rejects(changes, status):
    assert call("qw_experts_combine", COMBINE, **changes) == status


def test_nothing_to_do():
    assert call("qw_add_rms_norm", NORM, tokens=0) == OK
    assert call("qw_add_rms_norm_quantize", CODES, tokens=0, x=0, res=0, h=0) == OK
    for zero in (dict(m=0), dict(n=0)):
        assert call("qw_w8a16_linear_path", LINEAR, **zero) == OK
        assert call("qw_w8a8_linear_path", A8, **zero) == OK
    assert call("qw_w8a8_linear_path", A8, m=0, sx=0) == OK
    assert call("qw_w8a16_experts_path", EXPERTS, entries=0) == OK
    assert call("qw_w8a16_experts_path", EXPERTS, n=0) == OK
    assert call("qw_experts_combine", COMBINE, tokens=0) == OK
    assert call("qw_experts_combine", COMBINE, n=0) == OK


def test_workspaces():
    lib = qw.library()
    assert lib.qw_route_experts_workspace(0, 64, 8) == 0
    assert lib.qw_route_experts_workspace(64, 64, 8) == 64 * 4
    assert lib.qw_route_experts_workspace(65, 61, 8) == 2 * 64 * 4
    assert lib.qw_route_experts_workspace(1 << 20, 512, 8) <= 256 * 512 * 4
    for bad in ((-1, 64, 8), (1, 0, 8), (1, 513, 8), (1, 64, 0), (1, 64, 65), (1 << 31, 8, 1)):
        assert lib.qw_route_experts_workspace(*bad) == -1
    for f in (lib.qw_w8a16_linear_workspace, lib.qw_w8a8_linear_workspace):
        assert f(0, 64, 64, 0) == 0 and f(4, 64, 64, 1) == 0 and f(2048, 4096, 4096, 0) == 0
        assert f(2048, 4096, 16384, 0) > 0
        for bad in ((-1, 64, 64, 0), (1, -1, 64, 0), (1, 64, 0, 0), (1, 64, 24, 0), (1, 63, 64, 1), (1, 64, 64, 2), (1 << 31, 64, 64, 0)):
            assert f(*bad) == -1
    assert lib.qw_w8a8_linear_workspace(64, 64, 131088, 0) == -1


def meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device=META)


I8, I32, F32, BF16 = torch.int8, torch.int32, torch.float32, torch.bfloat16


def test_binding_checks_the_norm():
    check = qw.ff._validate_norm
    x, w = meta(3, 64), meta(64)
    assert check(x, w, x, False, None, META)[:4] == (0, 3, 64, 64)
    assert check(meta(3, 200)[:, 8:72], w, x, True, None, META)[3] == 200
    for bad in (dict(x=meta(3, 64, dtype=F32)), dict(x=meta(64)), dict(x=meta(64, 3).t()), dict(x=meta(3, 68)[:, :64]), dict(weight=meta(63)),
                dict(weight=meta(64, dtype=BF16)), dict(residual=meta(4, 64)), dict(residual=meta(3, 64, dtype=BF16)),
                dict(out=(meta(3, 64),)), dict(out=(meta(3, 32), None)), dict(out=(None, meta(3, 63))), dict(out=(None, None, None)),
                dict(quantize=True, out=(meta(3, 64), None, None)), dict(residual=None, out=(None, meta(3, 64)))):
        args = dict(x=x, weight=w, residual=x, quantize=False, out=None, device=META)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            check(**args)


def test_binding_checks_linear():
    check = qw.ff._validate_linear
    good = dict(x=meta(5, 64), q=meta(32, 64, dtype=I8), scales=meta(32), bias=meta(32), gated=False, residual=meta(5, 32), out=None,
                dtype=torch.float16, device=META)
    assert check(**good)[:3] == (5, 32, 64)
    assert check(**dict(good, gated=True, residual=meta(5, 16)))[3].shape == (5, 16)
    a8 = dict(good, x=meta(5, 64, dtype=I8), sx=meta(5), dtype=BF16, bias=meta(32, dtype=BF16), residual=meta(5, 32, dtype=BF16))
    assert check(**a8)[3].dtype == BF16
    for bad in (dict(x=meta(5, 64, dtype=BF16)), dict(x=meta(5, 48)), dict(x=meta(64, 5).t()), dict(q=meta(32, 64)), dict(scales=meta(31)),
                dict(bias=meta(16)), dict(bias=meta(32, dtype=F32)), dict(residual=meta(5, 16)), dict(gated=True), dict(out=meta(4, 32)),
                dict(gated=True, q=meta(31, 64, dtype=I8), scales=meta(31), bias=meta(31), residual=None), dict(out=meta(5, 32, dtype=BF16)),
                dict(x=torch.empty(5, 64, dtype=torch.float16))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))
    for bad in (dict(sx=meta(4)), dict(sx=meta(5, dtype=F32)), dict(bias=meta(32)), dict(x=meta(5, 64))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(a8, **bad))
    for name in ("swish", 3, ["relu"]):
        with pytest.raises(ValueError):
            qw.ff._activation(name)


def test_binding_checks_the_route():
    check = qw.ff._validate_route
    good = dict(logits=meta(9, 24), top_k=3, bias=meta(24, dtype=F32), groups=4, top_groups=2, device=META)
    assert check(**good) == (9, 24)
    for bad in (dict(logits=meta(9, 24, dtype=I32)), dict(logits=meta(24)), dict(logits=meta(24, 9).t()), dict(logits=meta(9, 513), bias=None, groups=1,
                top_groups=1), dict(logits=meta(9, 0), bias=None), dict(top_k=0), dict(top_k=65), dict(bias=meta(24)), dict(bias=meta(23, dtype=F32)),
                dict(groups=5), dict(groups=0), dict(top_groups=5), dict(top_groups=0)):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))


def route(tokens, top_k, experts, **changes):
    parts = dict(ids=meta(tokens, top_k, dtype=I32), weights=meta(tokens, top_k, dtype=F32), offsets=meta(experts + 1, dtype=I32),
                 rows=meta(tokens * top_k, dtype=I32), places=meta(tokens, top_k, dtype=I32))
    parts.update(changes)
    return qw.ExpertRoute(**parts)


def test_binding_checks_the_experts():
    check = qw.ff._validate_experts
    good = dict(x=meta(6, 64), q=meta(5, 32, 64, dtype=I8), scales=meta(5, 32), route=route(6, 2, 5), bias=meta(5, 32), gated=True, gather=True,
                out=None, device=META)
    assert check(**good)[:6] == (6, 64, 2, 12, 5, 32) and check(**good)[6].shape == (12, 16)
    assert check(**dict(good, x=meta(12, 64), gather=False))[0] == 12
    for bad in (dict(x=meta(12, 64)), dict(gather=False), dict(x=meta(6, 48)), dict(q=meta(32, 64, dtype=I8)), dict(q=meta(5, 31, 64, dtype=I8)),
                dict(scales=meta(5, 31)), dict(bias=meta(32)), dict(route=route(6, 2, 4)), dict(route=route(6, 2, 5, rows=meta(11, dtype=I32))),
                dict(route=route(6, 2, 5, offsets=meta(6))), dict(out=meta(12, 32)), dict(x=meta(6, 64, dtype=BF16))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))
    check = qw.ff._validate_combine
    good = dict(y=meta(12, 40), route=route(6, 2, 5), residual=meta(6, 40), out=None, device=META)
    assert check(**good)[:3] == (6, 2, 40)
    for bad in (dict(y=meta(11, 40)), dict(y=meta(12, 40, dtype=BF16)), dict(route=route(6, 2, 5, weights=meta(6, 2))), dict(residual=meta(12, 40)),
                dict(route=route(6, 2, 5, places=meta(6, 2))), dict(out=meta(6, 39)), dict(residual=meta(6, 40, dtype=F32))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))


def test_calls_refuse_host_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.float16)
    q, s = torch.zeros(32, 64, dtype=I8), torch.zeros(32, dtype=torch.float16)
    r = qw.ExpertRoute(torch.zeros(2, 1, dtype=I32), torch.zeros(2, 1), torch.zeros(6, dtype=I32), torch.zeros(2, dtype=I32),
                       torch.zeros(2, 1, dtype=I32))
    for f in (lambda: qw.add_rms_norm(x, w), lambda: qw.w8a16_linear(x, q, s), lambda: qw.w8a8_linear(x.to(I8), x[:, 0].contiguous(), q, s),
              lambda: qw.route_experts(x, 2), lambda: qw.w8a16_experts(x, q[None], s[None], r), lambda: qw.experts_combine(x, r)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for f in (lambda: qw.add_rms_norm(None, w), lambda: qw.w8a16_linear([1], q, s), lambda: qw.route_experts(3, 2), lambda: qw.experts_combine(None, r)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError, match="scoring"):
        qw.route_experts(x, 2, scoring="tanh")
