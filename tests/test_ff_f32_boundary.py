"""The experts' calls with fp32 entries without a GPU: what the C ABI and the
binding reject."""

import pytest

torch = pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")
import test_ff_boundary as ff  # noqa: E402
import test_ff_host as host  # noqa: E402

devices, second = host.devices, host.second
OK, INVALID, MISALIGNED, UNSUPPORTED = ff.OK, ff.INVALID, ff.MISALIGNED, ff.UNSUPPORTED
P, meta, F32 = ff.P, ff.meta, torch.float32


@pytest.mark.parametrize("changes,status", [
    (dict(act=9), INVALID), (dict(n=63), INVALID), (dict(gather=0), INVALID), (dict(path=1), INVALID), (dict(path=2, tile=128128), INVALID),
    (dict(y=0), INVALID), (dict(k=120), UNSUPPORTED), (dict(entries=1 << 31), UNSUPPORTED), (dict(y=P[6] + 8), MISALIGNED),
    (dict(y=P[1] - 40 * 32 * 4 + 16), INVALID),  # (its end within the weights: twice as far as in fp16)
    (dict(y=P[4] - 40 * 32 * 4 + 16), INVALID), (dict(entries=0), OK), (dict(n=0), OK),
])
def test_experts_rejects(changes, status):
    assert ff.call("qw_w8a16_experts_f32", ff.EXPERTS, **changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(entries=-1), INVALID), (dict(top_k=0), INVALID), (dict(y=0), INVALID), (dict(out=0), INVALID), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(y=P[0] + 8), MISALIGNED), (dict(out=P[0] + 40 * 64 * 4 - 16), INVALID), (dict(out=P[3] + 16), INVALID), (dict(tokens=0), OK),
])
def test_combine_rejects(changes, status):
    assert ff.call("qw_experts_combine_f32", ff.COMBINE, **changes) == status


def test_binding():
    check = qw.ff._validate_experts
    good = dict(x=meta(6, 64), q=meta(5, 32, 64, dtype=torch.int8), scales=meta(5, 32), route=ff.route(6, 2, 5), bias=None, gated=True,
                gather=True, out=None, device=ff.META, dtype=F32)
    assert check(**good)[6].dtype == F32
    assert check(**dict(good, out=meta(12, 16, dtype=F32)))[6].dtype == F32
    for bad in (dict(dtype=torch.bfloat16), dict(dtype="float32"), dict(out=meta(12, 16)), dict(dtype=torch.float16, out=meta(12, 16, dtype=F32)),
                dict(out=meta(12, 32, dtype=F32))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))
    check = qw.ff._validate_combine
    good = dict(y=meta(12, 40, dtype=F32), route=ff.route(6, 2, 5), residual=meta(6, 40), out=None, device=ff.META)
    assert check(**good)[3].dtype == torch.float16
    for bad in (dict(y=meta(12, 40, dtype=torch.float64)), dict(y=meta(11, 40, dtype=F32)), dict(out=meta(6, 40, dtype=F32))):
        with pytest.raises((TypeError, ValueError)):
            check(**dict(good, **bad))


@pytest.mark.parametrize("call", [
    lambda: qw.w8a16_experts(second((4, 32)), second((3, 8, 32), torch.int8), second((3, 8)), host.route_on_second(), dtype=F32),
    lambda: qw.w8a16_experts(second((8, 32)), second((3, 8, 32), torch.int8), second((3, 8)), host.route_on_second(), gather=False,
                             out=second((8, 8), F32), dtype=F32),
    lambda: qw.experts_combine(second((8, 16), F32), host.route_on_second(), residual=second((4, 16))),
])
def test_operands_on_another_device_than_the_current_one(devices, call):
    call()
