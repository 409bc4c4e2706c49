"""The host code of the KV cache calls under the host sanitizers (CPU only): the
library built as for the other calls' run, and the boundary, size and binding
tests of these against it."""

import os
import tempfile

import pytest

pytest.importorskip("torch")
san = pytest.importorskip("test_sanitizers")

pytestmark = pytest.mark.slow


def test_kv_host_code_under_address_and_ub_sanitizers():
    rt = san._clang_asan_runtime()
    if rt is None or not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("no hipcc / clang sanitizer runtime")
    from int8_weight_quantized_amd import build as qwbuild
    host_only = [f for flag in san.SAN for f in ("-Xarch_host", flag)]
    with tempfile.TemporaryDirectory() as tmp:
        lib = qwbuild.build(extra=host_only, build_dir=os.path.join(tmp, "obj"), output=os.path.join(tmp, "libqw_san.so"))
        out = san._run_child(["tests/test_kv_boundary.py", "tests/test_kv_sizes.py", "tests/test_kv_host.py"],
                             {"QW_LIBRARY": lib, "LD_PRELOAD": rt}, tmp)
    assert " passed" in out
