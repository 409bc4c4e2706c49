"""Feed-forward calls of so many rows or channels that one grid does not hold a
thread for each piece of work (2^32 threads)."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16 = torch.float16
GPU = "cuda:0"


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.get_device_properties(0).total_memory < (160 << 30):
        pytest.skip("needs 160 GiB")
    yield
    torch.cuda.empty_cache()


def ints(seed, shape, top, dtype):
    g = torch.Generator(device=GPU)
    g.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=GPU, dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_rows(residual, quantize):
    """256 threads a row: 2^24 rows are 2^32 threads.  Every row as in calls of
    parts of them."""
    T, K = (1 << 24) + 37, 16
    print("norm", T, K, residual, quantize, flush=True)
    x = ints(1, (T, K), 100, F16)
    r = ints(2, (T, K), 100, F16) if residual else None
    w = torch.linspace(0.5, 2, K, device=GPU).half()
    whole = qw.add_rms_norm(x, w, residual=r, quantize=quantize)
    cut = [0, 5000001, (1 << 23) - 1, (1 << 23) + 3, T - 1, T]
    for a, b in zip(cut, cut[1:]):
        part = qw.add_rms_norm(x[a:b], w, residual=None if r is None else r[a:b], quantize=quantize)
        for one, other in zip(whole, part):
            assert torch.equal(one[a:b], other)
    h = x.double() if r is None else x.double() + r.double()
    y = h * w.double() / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    if quantize:
        got = whole[0].double() * whole[1].double()[:, None]
        assert ((got - y).abs() <= 0.51 * whole[1].double()[:, None]).all()
    else:
        assert ((whole[0].double() - y).abs() <= 2.0 ** -10.9 * y.abs() + 2.0 ** -24).all()


@pytest.mark.parametrize("f32", [False, True])
def test_combine_pieces(f32):
    """A thread for 8 columns of a token: 2^26 tokens of 512 are 2^32 threads.
    The tokens' places are a few rows."""
    T, n, rows = (1 << 26) + 5, 512, 64
    print("combine", T, n, f32, flush=True)
    y = ints(3, (rows, n), 100, torch.float32 if f32 else F16)
    g = torch.Generator(device=GPU)
    g.manual_seed(4)
    places = torch.randint(-1, rows, (T, 1), generator=g, device=GPU, dtype=torch.int32)
    weights = torch.full((T, 1), 0.5, device=GPU)
    out = torch.full((T, n), 7.0, dtype=F16, device=GPU)
    call = qw.library().qw_experts_combine_f32 if f32 else qw.library().qw_experts_combine
    st = call(y.data_ptr(), rows, places.data_ptr(), weights.data_ptr(), T, 1, None, out.data_ptr(), n,
              torch.cuda.current_stream().cuda_stream)
    assert st == 0, qw.status_string(st)
    for at in range(0, T, 1 << 22):
        p = places[at:at + (1 << 22), 0].long()
        want = torch.where((p < 0)[:, None], 0.0, y.float()[p.clamp(min=0)] * 0.5)
        assert torch.equal(out[at:at + (1 << 22)].float(), want)


@pytest.mark.parametrize("m,n,gated,a8", [(5, (1 << 29) + 64, False, False), (5, (1 << 29) + 64, False, True),
                                          (20, (1 << 30) + 128, False, False), (5, (1 << 30) + 128, True, False)])
def test_channels(m, n, gated, a8):
    """Eight (or, with 128 rows a workgroup, four) threads a channel where waves
    share the activations."""
    k = 16
    print("channels", m, n, gated, a8, flush=True)
    q = ints(5, (n, k), 127, torch.int8)
    s = torch.full((n,), 2.0 ** -6, dtype=F16, device=GPU)
    x = ints(6, (m, k), 3, torch.int8 if a8 else F16)
    columns = n // 2 if gated else n
    y = torch.full((m, columns), float("nan"), dtype=F16, device=GPU)
    if a8:
        qw.w8a8_linear(x, torch.ones(m, dtype=F16, device=GPU), q, s, out=y)
    else:
        qw.w8a16_linear(x, q, s, activation="relu" if gated else None, gated=gated, out=y)
    for c in range(0, columns, 1 << 25):
        e = min(columns, c + (1 << 25))

        def product(lo):
            # (integers below 2^24 and powers of two: exact in fp32)
            return x.float() @ q[lo + c:lo + e].float().t() * 2.0 ** -6
        want = product(0).clamp(min=0) * product(columns) if gated else product(0)
        assert torch.equal(y[:, c:e], want.half())
