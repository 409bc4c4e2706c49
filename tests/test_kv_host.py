"""The binding of the KV cache calls between its checks and the library,
without a GPU."""

import threading

import pytest

torch = pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")
kv = qw.kv


def test_first_calls_from_two_threads(monkeypatch):
    """A call that begins while another thread's first one loads torch."""
    found = []

    def second():
        try:
            found.append(kv._dtype_code(torch.bfloat16, "q"))
            found.append(kv._raw_stream is not None)
        except Exception as e:  # noqa: BLE001
            found.append(e)

    class Codes(dict):
        begun = False

        def update(self, *args):
            if not Codes.begun:  # nothing is in it yet, in the first thread's call
                Codes.begun = True
                other = threading.Thread(target=second)
                other.start()
                other.join(30)
            super().update(*args)

    monkeypatch.setattr(kv, "_torch", None)
    monkeypatch.setattr(kv, "_raw_stream", None)
    monkeypatch.setattr(kv, "_codes", Codes())
    assert kv._dtype_code(torch.float16, "q") == 0
    assert found == [1, True]


class OnSecond(torch.Tensor):
    """A tensor that says it is on the second GPU."""

    @staticmethod
    def __new__(cls, data):
        return data.as_subclass(cls)

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


def second(shape, dtype=torch.float16):
    return OnSecond(torch.zeros(shape, dtype=dtype))


@pytest.fixture
def devices(monkeypatch):
    """Two GPUs, the first one current; the library notes which one is at each
    call."""
    now, calls = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *error):
            now[0] = self.before

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, now[0])) or 0

    empty, empty_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *a, **k: OnSecond(empty(*a, **dict(k, device="cpu"))))
    monkeypatch.setattr(torch, "empty_like", lambda t: OnSecond(empty(t.shape, dtype=t.dtype)))
    kv._load_torch()
    monkeypatch.setattr(kv, "_current_device", lambda: now[0], raising=False)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(qw, "_stream_of", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(qw, "library", Library)
    yield calls
    assert calls and now == [0]
    assert all(index == 1 for _, index in calls), calls


I32, F32, I8 = torch.int32, torch.float32, torch.int8


def cache_on_second():
    return (second((3, 2, 16, 64), I8), second((3, 2, 64, 16), I8), second((3, 2), F32), second((3, 2), F32))


@pytest.mark.parametrize("call", [
    lambda: qw.kv_plan(second(2, I32), second(2, I32), second((2, 3), I32), second(4, I32), 16, 5),
    lambda: qw.qk_norm_rope(second((5, 4, 64)), second((5, 2, 64)), second(5, I32), second((9, 16), F32), second((9, 16), F32)),
    lambda: qw.kv_write(second((5, 2, 64)), second((5, 2, 64)), second(5, I32), *cache_on_second()),
    lambda: qw.kv_read(second(5, I32), *cache_on_second()),
    lambda: qw.kv_attention(second((5, 4, 64)), *cache_on_second(), second((2, 3), I32), second(2, I32), second(3, I32), 3),
    lambda: qw.kv_attention_workspace(second((5, 4, 64)), cache_on_second()[0], second((2, 3), I32), 3),
    lambda: qw.quantize_weights(second((8, 32))),
    lambda: qw.quantize_weights_fixed_range(second((8, 32), F32), second(8, F32)),
    lambda: qw.quantize_weights_asym(second((8, 32), F32)),
    lambda: qw.w8a16_gemm(second((2, 32)), second((8, 32), I8), second(8)),
    lambda: qw.w8a16_gemm_tune(second((2, 32)), second((8, 32), I8), second(8)),
    lambda: qw.w8a16_gemm_asym(second((2, 32)), second((8, 32), I8), second(8), second(8, I8)),
    lambda: qw.w8a16_gemm_outliers(second((2, 32)), second((8, 32), I8), second(8), second((8, 1), I32), second((8, 1), F32)),
    lambda: qw.w8a8_gemm(second((2, 32), I8), second(2), second((8, 32), I8), second(8)),
    lambda: qw.w8a8_gemm_tile(second((2, 32), I8), second(2), second((8, 32), I8), second(8), qw.W8A8_TILES[0]),
    lambda: qw.w8a16_gemm_tile(second((2, 32)), second((8, 32), I8), second(8), qw.MFMA_TILES[0]),
])
def test_operands_on_another_device_than_the_current_one(devices, call):
    """The operands' device is current while the library launches on it."""
    call()
