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
