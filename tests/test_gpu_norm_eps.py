"""add_rms_norm with an eps that binary32 does not hold."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("eps", [1e-38, 1e-44, 1e-46, 1e-60, 1e-300, 5e-324])
def test_rows_of_zeros(eps, dtype):
    """0 / sqrt(eps) is 0; the other rows do not see so small an eps."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(6, 512, generator=gen, device="cuda").to(dtype)
    x[2], x[5] = 0, 0
    w = torch.ones(512, dtype=dtype, device="cuda")
    r = torch.zeros_like(x)
    for residual in (None, r):
        y, _ = qw.add_rms_norm(x, w, residual=residual, eps=eps)
        q, s, _ = qw.add_rms_norm(x, w, residual=residual, eps=eps, quantize=True)
        for row in (2, 5):
            assert torch.equal(y[row], r[row]) and not q[row].any() and s[row] == 0
        some = [0, 1, 3, 4]
        y0, _ = qw.add_rms_norm(x[some], w, eps=0.0)
        q0, s0, _ = qw.add_rms_norm(x[some], w, eps=0.0, quantize=True)
        assert torch.equal(y[some], y0) and torch.equal(q[some], q0) and torch.equal(s[some], s0)
