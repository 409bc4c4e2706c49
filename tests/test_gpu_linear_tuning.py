"""Which kernel w8a16_linear and w8a8_linear run with a tuning record of the plain
product: by the workspaces they ask for and by their bits, which differ between
kernels for sums that fp32 rounds."""

import pytest

torch = pytest.importorskip("torch")
import test_gpu_linear as linear  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16 = torch.float16


@pytest.fixture(autouse=True)
def clean_records():
    qw.tune_reset()
    yield
    qw.tune_reset()


def operands(seed, m, n, k):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(m, k, generator=gen, device="cuda")
    q, s = qw.quantize_weights(torch.randn(n, k, generator=gen, device="cuda") / k ** 0.5)
    return x.half(), q, s


def workspaces(m, n, k, gated=0):
    lib = qw.library()
    return lib.qw_w8a16_linear_workspace(m, n, k, gated), lib.qw_w8a8_linear_workspace(m, n, k, gated)


def tune_a8(x, q, s):
    qx, sx = qw.quantize_activations(x)
    y = torch.empty(len(x), len(q), dtype=F16, device="cuda")
    st = qw.w8a8_gemm_tune_raw(qx.data_ptr(), sx.data_ptr(), q.data_ptr(), s.data_ptr(), y.data_ptr(), *x.shape[:1], len(q), x.shape[1],
                               torch.cuda.current_stream().cuda_stream)
    assert st == 0, qw.status_string(st)
    return qx, sx


def test_a_record_takes_the_place_of_a_split():
    """256 x 1024 x 16384 splits by itself; a record names a kernel that does
    not, of its own type alone."""
    m, n, k = 256, 1024, 16384
    x, q, s = operands(1, m, n, k)
    before = workspaces(m, n, k)
    assert min(before) > 0
    qw.w8a16_gemm_tune(x, q, s)
    path, tile = qw.tuned_choice(m, n, k)
    print("w8a16", path, tile, flush=True)
    assert workspaces(m, n, k) == (0, before[1])
    forced = linear.call(x, None, q, s, None, None, path=path, tile=tile[0] * 1000 + tile[1] if tile else 0)
    assert torch.equal(qw.w8a16_linear(x, q, s), forced)
    assert workspaces(m + 8, n, k) == workspaces(m + 9, n, k) and workspaces(m, n, k - 16)[0] > 0  # (other buckets)
    qw.tune_reset()
    assert workspaces(m, n, k) == before
    split = qw.w8a16_linear(x, q, s)
    assert not torch.equal(split, forced)
    qx, sx = tune_a8(x, q, s)
    path, tile = qw.w8a8_tuned_choice(m, n, k)
    print("w8a8", path, tile, flush=True)
    assert workspaces(m, n, k) == (before[0], 0)
    assert torch.equal(qw.w8a16_linear(x, q, s), split)
    forced = linear.call(qx, sx, q, s, None, None, path=path, tile=tile[0] * 1000 + tile[1] if tile else 0)
    assert torch.equal(qw.w8a8_linear(qx, sx, q, s), forced)


@pytest.mark.parametrize("m,n,k,gated", [(3, 512, 4096, False), (6, 512, 1024, True), (1, 256, 9216, True), (1, 256, 4096, True)])
def test_a_kernel_that_the_epilogue_does_not_take(m, n, k, gated):
    """A record of the GEMV where it takes no epilogue: more than two rows, or gated
    with rows of more than 8192.  The skinny kernel runs."""
    x, q, s = operands(2, m, n, k)
    qw.w8a16_gemm_tune(x, q, s)
    path, tile = qw.tuned_choice(m, n, k)
    print("gemv", m, n, k, gated, path, tile, flush=True)
    if path == "gemv" and (m > 2 or (gated and k > 8192)):
        path = "skinny"
    forced = linear.call(x, None, q, s, None, None, act="silu", gated=gated, path=path, tile=tile[0] * 1000 + tile[1] if tile else 0)
    assert workspaces(m, n, k, int(gated))[0] == 0
    assert torch.equal(qw.w8a16_linear(x, q, s, activation="silu", gated=gated), forced)
