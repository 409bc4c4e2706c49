"""The binding of the feed-forward calls between its checks and the library,
without a GPU."""

import pytest

torch = pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")
host = pytest.importorskip("test_kv_host")

second, devices = host.second, host.devices
I8, I32, F32 = torch.int8, torch.int32, torch.float32


def route_on_second():
    return qw.ExpertRoute(second((4, 2), I32), second((4, 2), F32), second(4, I32), second(8, I32), second((4, 2), I32))


@pytest.mark.parametrize("call", [
    lambda: qw.add_rms_norm(second((2, 32)), second(32)),
    lambda: qw.add_rms_norm(second((2, 32)), second(32), residual=second((2, 32)), quantize=True),
    lambda: qw.add_rms_norm(second((2, 32)), second(32), out=(second((2, 32)), None)),
    lambda: qw.w8a16_linear(second((2, 32)), second((8, 32), I8), second(8)),
    lambda: qw.w8a16_linear(second((40, 32)), second((8, 32), I8), second(8), gated=True, residual=second((40, 4)), out=second((40, 4))),
    lambda: qw.w8a8_linear(second((40, 32), I8), second(40), second((8, 32), I8), second(8), dtype=torch.bfloat16),
    lambda: qw.route_experts(second((4, 3)), 2, bias=second(3, F32)),
    lambda: qw.w8a16_experts(second((4, 32)), second((3, 8, 32), I8), second((3, 8)), route_on_second()),
    lambda: qw.w8a16_experts(second((8, 32)), second((3, 8, 32), I8), second((3, 8)), route_on_second(), gather=False, out=second((8, 8))),
    lambda: qw.experts_combine(second((8, 16)), route_on_second(), residual=second((4, 16))),
])
def test_operands_on_another_device_than_the_current_one(devices, call):
    """The operands' device is current while the library launches on it."""
    call()


def test_a_route_is_needed(devices):
    for call in (lambda r: qw.w8a16_experts(second((4, 32)), second((3, 8, 32), I8), second((3, 8)), r),
                 lambda r: qw.experts_combine(second((8, 16)), r)):
        for bad in (None, 3, second((4, 2), I32)):
            with pytest.raises(TypeError, match="ExpertRoute"):
                call(bad)
        call(route_on_second())


def test_workspaces_are_asked_for(monkeypatch):
    """A product whose reduction the library splits takes the bytes it names;
    four rows and fewer never do, and are not asked about."""
    asked, given = [], []

    class Library:
        def qw_w8a16_linear_workspace(self, m, n, k, gated):
            asked.append((m, n, k, gated))
            return 4096 if k == 64 else 0

        def qw_w8a16_linear(self, *args):
            given.append(args[-3:-1])
            return 0

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: host.OnSecond(empty(*a, **dict(k, device="cpu"))))
    qw.kv._load_torch()
    monkeypatch.setattr(qw.kv, "_current_device", lambda: 1, raising=False)
    monkeypatch.setattr(qw.kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(qw, "library", Library)
    for m, k in ((4, 64), (5, 64), (5, 32)):
        qw.w8a16_linear(second((m, k)), second((8, k), I8), second(8), gated=True)
    assert asked == [(5, 8, 64, 1), (5, 8, 32, 1)]
    assert given[0] == given[2] == (None, 0) and given[1][0] and given[1][1] == 4096
