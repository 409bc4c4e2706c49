"""The experts' products in fp32 and their sum: nothing is rounded in between."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import assert_rounded, integers, made_route, scale16  # noqa: E402
import test_gpu_experts as fp16  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

F16, F32 = torch.float16, torch.float32


def check(seed, ids, experts, n, k, act=None, gated=False, gather=True, bias=True, path="auto", tile=0):
    """The fp16 call on one kernel (checked there), and the fp32 call on the same."""
    x, q, s, b, route, y16 = fp16.check(seed, ids, experts, n, k, act, gated, gather, bias, path, tile)
    want, off = fp16.want_of(x, q, s, b, route, act, gated, gather)
    y = torch.full(want.shape, 55.0, dtype=F32, device="cuda")
    st = qw.library().qw_w8a16_experts_f32(
        x.data_ptr(), x.shape[0], int(gather), q.data_ptr(), s.data_ptr(), None if b is None else b.data_ptr(),
        qw.ACTIVATIONS[act], int(gated), route.offsets.data_ptr(), route.rows.data_ptr(), len(y), len(ids[0]), y.data_ptr(), experts,
        n, k, qw.PATHS[path], tile, torch.cuda.current_stream().cuda_stream)
    assert st == 0, qw.status_string(st)
    assert_rounded(y, want, off)
    assert torch.equal(y.half(), y16)
    assert not y[route.offsets[-1]:].any()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 1, 1, 16, 16), (1, 8, 2, 64, 64), (7, 5, 3, 34, 48), (32, 64, 8, 130, 272),
                                                      (40, 3, 2, 256, 1040), (3, 512, 4, 32, 32), (64, 16, 1, 528, 128), (9, 4, 2, 662, 96)])
def test_skinny(tokens, experts, top_k, n, k, gather, gated):
    check(1, fp16.ids_of(2, tokens, experts, top_k, none=0.2), experts, n, k, "silu", gated, gather, path="skinny")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", fp16.TILES)
@pytest.mark.parametrize("tokens,experts,top_k,n,k,none", [(1, 2, 1, 2, 16, 0.0), (90, 4, 2, 260, 80, 0.1), (600, 3, 2, 518, 208, 0.3),
                                                           (257, 1, 1, 300, 64, 0.0), (700, 9, 4, 512, 400, 0.0), (100, 3, 2, 662, 96, 0.0)])
def test_tiles(tokens, experts, top_k, n, k, none, tile, gated):
    ids = fp16.ids_of(3, tokens, experts, top_k, none)
    check(4, ids, experts, n, k, "silu" if gated else "relu", gated, True, path="mfma", tile=tile)
    check(5, ids, experts, n, k, None, gated, False, bias=False, path="mfma", tile=tile)


@pytest.mark.parametrize("tile", [256256, 128064])
def test_odd_columns(tile):
    check(11, fp16.ids_of(12, 100, 3, 2), 3, 331, 96, "gelu", path="mfma", tile=tile)
    check(15, fp16.ids_of(16, 9, 3, 2), 3, 331, 96, path="skinny")


@pytest.mark.parametrize("path,tile", [("skinny", 0), ("mfma", 256256), ("mfma", 256064)])
def test_uneven_experts(path, tile):
    for ids in ([[0]] * 300, [[5]] * 300, [[-1]] * 300, [[0]] * 256 + [[3]] * 64 + [[5]] * 16 + [[-1]], [[2]] * 255 + [[3]] * 257,
                [[-1]] * 40 + [[1]] * 15 + [[2]] * 17):
        check(10, ids, 6, 64, 96, path=path, tile=tile)


def sum64(want, off, route, residual):
    """The sum over a token's entries in 64 bits, and how far fp32 may be off."""
    total, size = fp16.combine64(want, route, residual)
    places = route.places.long()
    each = torch.where((places < 0)[:, :, None], 0.0, off[places.clamp(min=0)]) * route.weights.double()[:, :, None]
    return total, size + each.sum(1)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 8, 2, 40, 64), (32, 64, 8, 512, 256), (500, 6, 4, 331, 128), (64, 4, 1, 8, 16)])
def test_one_rounding(tokens, experts, top_k, n, k, residual):
    """Product and sum, against 64 bits of both: the only rounding to 16 bits is
    the sum's."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(30)
    w = torch.rand(tokens, top_k, generator=gen, device="cuda")
    route = made_route(fp16.ids_of(31, tokens, experts, top_k, none=0.1), w)(experts)
    x, q, s, b = fp16.operands(32, tokens * top_k, experts, n, k)
    r = torch.randn(tokens, n, generator=gen, device="cuda").half() if residual else None
    want, off = fp16.want_of(x, q, s, b, route, None, False, False)
    total, off = sum64(want, off, route, r)
    y = qw.w8a16_experts(x, q, s, route, bias=b, gather=False, dtype=F32)
    assert y.dtype is F32
    assert_rounded(qw.experts_combine(y, route, residual=r), total, off)
    out = torch.empty_like(y)
    with pytest.raises(TypeError):
        qw.w8a16_experts(x, q, s, route, bias=b, gather=False, out=out)  # (fp16 unless it is asked for)
    assert qw.w8a16_experts(x, q, s, route, bias=b, gather=False, out=out, dtype=F32) is out and torch.equal(out, y)


def test_entries_beyond_fp16():
    """Entries of up to some 2^18 that cancel, and that their weights make small."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(33)
    ids = [[0, 1]] * 20
    w = torch.full((20, 2), 2.0 ** -6, device="cuda")
    route = made_route(ids, w)(2)
    x = torch.ones(40, 64, dtype=F16, device="cuda")
    q = integers(gen, (2, 24, 64), 127, torch.int8)
    q[1] = -q[0]
    s = torch.full((2, 24), 256.0, dtype=F16, device="cuda")
    y = qw.w8a16_experts(x, q, s, route, gather=False, dtype=F32)
    v = q.double().sum(2) * 256
    assert v.abs().max() > 65504
    assert torch.equal(y.double(), v.repeat_interleave(20, 0))
    assert not qw.experts_combine(y, route).any()
    route.weights[:, 1] = 2.0 ** -7
    assert_rounded(qw.experts_combine(y, route), (v[0] * 2.0 ** -7).expand(20, 24), torch.zeros(20, 24, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("tokens,experts,top_k,n", [(1, 1, 1, 8), (1, 8, 2, 1), (5, 8, 8, 333), (64, 64, 6, 2048), (30, 100, 19, 40), (3000, 16, 2, 24)])
def test_combine(tokens, experts, top_k, n):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(34)
    w = torch.rand(tokens, top_k, generator=gen, device="cuda")
    route = made_route(fp16.ids_of(35, tokens, experts, top_k, none=0.2), w)(experts)
    y = torch.randn(tokens * top_k, n, generator=gen, device="cuda")
    y[route.offsets[-1]:] = float("nan")  # (never read)
    r = torch.randn(tokens, n, generator=gen, device="cuda").half()
    want, off = fp16.combine64(y, route, r)
    got = qw.experts_combine(y, route, residual=r)
    assert_rounded(got, want, off)
    assert qw.experts_combine(y, route, residual=r, out=r) is r and torch.equal(r, got)


def test_replayed_graph():
    route = made_route(fp16.ids_of(36, 12, 4, 2))(4)
    x, q, s, b = fp16.operands(37, 24, 4, 64, 96)
    xs = [fp16.operands(38 + i, 24, 4, 64, 96)[0] for i in range(4)]
    at = x.clone()

    def step():
        return qw.experts_combine(qw.w8a16_experts(at, q, s, route, bias=b, gather=False, dtype=F32), route)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for v in xs:
        at.copy_(v)
        graph.replay()
        assert torch.equal(out, step())


def test_outputs_beyond_four_gigabytes():
    if torch.cuda.get_device_properties(0).total_memory < (64 << 30):
        pytest.skip("needs 64 GiB")
    tokens, E, n, k = 300000, 2, 8192, 32
    route = qw.route_experts(torch.zeros(tokens, E, device="cuda"), E)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(39)
    x, q = integers(gen, (tokens * E, k), 3, F16), integers(gen, (E, n, k), 127, torch.int8)
    s = scale16(gen, (E, n), 2.0 ** -6)
    y = qw.w8a16_experts(x, q, s, route, gather=False, dtype=F32)
    out = qw.experts_combine(y, route)
    for t in (0, 1, tokens // 2 + 7, tokens - 1):
        v = [(q[e].double() @ x[t + e * tokens].double()) * s[e].double() for e in range(E)]
        for e in range(E):
            # (sums of integers are exact, the scaled one is rounded once)
            assert_rounded(y[t + e * tokens], v[e], torch.zeros_like(v[e]))
        assert_rounded(out[t], (v[0] + v[1]) / 2, 2.0 ** -23 * (v[0].abs() + v[1].abs()))
