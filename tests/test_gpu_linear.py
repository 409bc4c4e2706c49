"""w8a16_linear and w8a8_linear against 64 bits, on every kernel and tile.

The activations are small integers and the codes int8, so that every sum is
exact in fp32; what is left is the epilogue and one rounding."""

import pytest

torch = pytest.importorskip("torch")
from ff_reference import assert_rounded, integers, linear64, scale16  # noqa: E402

pytestmark = pytest.mark.gpu
qw = pytest.importorskip("int8_weight_quantized_amd")

PATHS = qw.PATHS
F16, BF16 = torch.float16, torch.bfloat16


def operands(seed, m, n, k, a8=False, dtype=F16, bias=True, residual=True, gated=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = integers(gen, (m, k), 127 if a8 else 4, torch.int8 if a8 else F16)
    sx = scale16(gen, (m,), 2.0 ** -6) if a8 else None
    q = integers(gen, (n, k), 127, torch.int8)
    # v of a few units, so that the activations bend
    s = scale16(gen, (n,), 2.0 ** -7 / k ** 0.5 if not a8 else 2.0 ** -7 / k ** 0.5)
    b = torch.randn(n, generator=gen, device="cuda").to(dtype) if bias else None
    r = (4 * torch.randn(m, n // 2 if gated else n, generator=gen, device="cuda")).to(dtype) if residual else None
    return x, sx, q, s, b, r


def call(x, sx, q, s, b, r, act=None, gated=False, dtype=F16, path="auto", tile=0, out=None, splits=1):
    print("linear", tuple(x.shape), tuple(q.shape), "w8a8" if sx is not None else "w8a16", act, gated, dtype, path, tile, splits, flush=True)
    (m, k), n = x.shape, q.shape[0]
    y = torch.full((m, n // 2 if gated else n), 77.0, dtype=dtype, device="cuda") if out is None else out
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    lib = qw.library()
    size = -(-m // 256) * -(-n // 256) * 262144 * splits if splits > 1 else 0
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    if sx is None:
        st = lib.qw_w8a16_linear_path(p(x), p(q), p(s), p(b), qw.ACTIVATIONS[act], int(gated), p(r), p(y), m, n, k, PATHS[path],
                                      tile, splits, p(ws), size, stream)
    else:
        st = lib.qw_w8a8_linear_path(p(x), p(sx), p(q), p(s), p(b), qw.ACTIVATIONS[act], int(gated), p(r),
                                     1 if dtype == BF16 else 0, p(y), m, n, k, PATHS[path], tile, splits, p(ws), size, stream)
    assert st == 0, qw.status_string(st)
    return y


def check(seed, m, n, k, a8=False, dtype=F16, act=None, gated=False, bias=True, residual=True, path="auto", tile=0,
          splits=1):
    ops = operands(seed, m, n, k, a8, dtype, bias, residual, gated)
    x, sx, q, s, b, r = ops
    want, off = linear64(x, q, s, b, act, gated, r, sx)
    assert_rounded(call(*ops, act, gated, dtype, path, tile, splits=splits), want, off)


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("path,m,n,k", [("gemv", 1, 130, 1008), ("gemv", 2, 96, 4096), ("skinny", 5, 136, 208),
                                        ("mfma", 70, 264, 144)])
def test_activations(path, m, n, k, act, gated):
    check(1, m, n, k, act=act, gated=gated, path=path)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", [None, "gelu", "silu"])
@pytest.mark.parametrize("path,m,n,k", [("skinny", 5, 136, 208), ("mfma", 70, 264, 144)])
def test_activations_w8a8(path, m, n, k, act, dtype):
    check(2, m, n, k, a8=True, dtype=dtype, act=act, path=path)
    check(3, m, n, k, a8=True, dtype=dtype, act=act, path=path, gated=True)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 1024), (2, 3008), (1, 5120), (2, 6144), (1, 8192), (2, 8176)])
def test_gemv(m, k, gated):
    check(4, m, 46, k, act="silu", gated=gated, path="gemv")
    check(5, m, 2 * 2049 if gated else 2049, k, gated=gated, path="gemv", bias=False)  # more columns than waves


@pytest.mark.parametrize("m", [1, 2])
def test_gemv_long_rows(m):
    check(6, m, 133, 9232, act="gelu", path="gemv")
    check(7, m, 64, 13696, path="gemv", bias=False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (3, 34, 48), (16, 64, 64), (17, 30, 2064), (32, 258, 2048), (33, 512, 1040), (7, 8224, 272),
                                   (64, 4098, 128), (32, 12546, 2048), (20, 8190, 2064)])
def test_skinny(m, n, k, a8, gated):
    check(8, m, n, k, a8=a8, act="silu" if gated else None, gated=gated, path="skinny", dtype=BF16 if a8 and gated else F16)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("m,n,k", [(5, 12290, 16), (16, 12346, 272), (9, 12354, 4112), (8, 24706, 528), (16, 24578, 48), (17, 24600, 2048),
                                   (32, 24578, 2064), (24, 12354, 4112), (12, 33026, 80), (31, 33002, 2304)])
def test_skinny_wide(m, n, k, a8, gated):
    """Many weight rows: waves that share the activations, one and two tiles of
    them, parts of k of different lengths or none, the last row block cut off."""
    check(21, m, n, k, a8=a8, act="silu" if gated else None, gated=gated, path="skinny", dtype=BF16 if a8 and gated else F16)


TILES = [256256, 256128, 256064, 128128, 128064]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(1, 2, 16), (300, 518, 208), (257, 264, 64), (130, 1026, 320), (256, 512, 400), (515, 300, 1088)])
def test_tiles(m, n, k, tile, gated):
    check(9, m, n, k, act="silu" if gated else "relu", gated=gated, path="mfma", tile=tile)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", [t for t in TILES if t != 128128])
@pytest.mark.parametrize("m,n,k", [(1, 2, 16), (300, 518, 208), (130, 1026, 320), (512, 512, 384)])
def test_tiles_w8a8(m, n, k, tile, gated):
    check(10, m, n, k, a8=True, act="silu" if gated else None, gated=gated, path="mfma", tile=tile)
    check(11, m, n, k, a8=True, dtype=BF16, gated=gated, path="mfma", tile=tile, bias=False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("m,n,k,splits", [(1, 2, 128, 2), (300, 518, 208, 3), (257, 264, 400, 2), (512, 1024, 1088, 8), (130, 1026, 4112, 5),
                                          (256, 256, 640, 10), (700, 300, 2000, 7)])
def test_split(m, n, k, splits, a8, gated):
    check(24, m, n, k, a8=a8, act="silu" if gated else "gelu", gated=gated, path="mfma", tile=256256, splits=splits)
    check(25, m, n, k, a8=a8, dtype=BF16 if a8 else F16, bias=False, residual=splits % 2 == 0, gated=gated, path="mfma", tile=256256,
          splits=splits)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("m,n,k,splits", [(1, 2, 128, 2), (5, 66, 400, 3), (16, 264, 1088, 8), (17, 130, 2064, 5), (32, 514, 4112, 4), (40, 70, 512, 8),
                                          (9, 1024, 8192, 8), (31, 192, 4096, 64)])
def test_skinny_parts(m, n, k, splits, a8, gated):
    check(22, m, n, k, a8=a8, act="silu" if gated else "relu", gated=gated, path="skinny", splits=splits, dtype=BF16 if a8 and gated else F16)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", [(9, 1024, 16400), (16, 4098, 8192), (32, 2050, 4096), (32, 8192, 4112)])
def test_skinny_parts_by_itself(m, n, k, gated):
    """Few rows, few channels and long rows are split, and the parts change the
    sum by fp32's roundings alone (here: not at all)."""
    assert qw.library().qw_w8a16_linear_workspace(m, n, k, int(gated)) > 0
    x, _, q, s, b, r = operands(23, m, n, k, gated=gated)
    split = qw.w8a16_linear(x, q, s, bias=b, activation="silu", gated=gated, residual=r)
    whole = call(x, None, q, s, b, r, "silu", gated, path="skinny")
    assert torch.equal(split, whole)


@pytest.mark.parametrize("m,n,k", [(512, 1024, 8192), (250, 520, 13696), (700, 2048, 9232)])
def test_split_by_itself(m, n, k):
    """Sizes that the calls split on their own."""
    x, _, q, s, b, r = operands(26, m, n, k)
    want, off = linear64(x, q, s, b, "silu", False, r)
    assert_rounded(qw.w8a16_linear(x, q, s, bias=b, activation="silu", residual=r), want, off)
    x, sx, q, s, b, r = operands(27, m, n, k, a8=True, dtype=BF16, gated=True)
    want, off = linear64(x, q, s, b, "silu", True, r, sx)
    assert_rounded(qw.w8a8_linear(x, sx, q, s, bias=b, activation="silu", gated=True, residual=r), want, off)


@pytest.mark.parametrize("tile", TILES)
def test_odd_columns(tile):
    check(12, 200, 331, 96, act="gelu", path="mfma", tile=tile)
    check(13, 200, 2 * 331, 96, act="gelu_tanh", gated=True, path="mfma", tile=tile)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("path,tile", [("gemv", 0), ("skinny", 0), ("mfma", 256256), ("mfma", 256128), ("mfma", 128064)])
def test_each_part_alone(path, tile, bias, residual):
    m = 2 if path == "gemv" else 40
    check(14, m, 256, 128, bias=bias, residual=residual, path=path, tile=tile)
    check(15, m, 256, 128, bias=bias, residual=residual, path=path, tile=tile, gated=True, act="silu")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("path,tile,m", [("gemv", 0, 2), ("skinny", 0, 30), ("mfma", 256256, 300), ("mfma", 256064, 300)])
def test_residual_in_place(path, tile, m, gated):
    x, sx, q, s, b, r = operands(16, m, 520, 336, gated=gated)
    want = call(x, sx, q, s, b, r, "silu", gated, path=path, tile=tile)
    got = call(x, sx, q, s, b, r, "silu", gated, path=path, tile=tile, out=r)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m,n,k", [(1, 4608, 4096), (2, 512, 4096), (8, 4608, 4096), (16, 1024, 1024), (48, 4608, 1024), (129, 4096, 1024),
                                   (700, 4608, 512)])
def test_auto_matches_the_plain_product(m, n, k):
    """Without bias, activation and residual: w8a16_gemm's result.  The plain
    MFMA kernels round a sum times its scale to fp16 in one step, the epilogue
    to fp32 and then to fp16: either is within 2^-11 + 2^-23 of the exact
    product, so they are at most twice that, and one fp16 step, apart."""
    def near(a, b):
        d, b = (a.double() - b.double()).abs(), b.double().abs()
        assert (d <= 2 * (2.0 ** -11 + 2.0 ** -23) * b * (1 + 2.0 ** -10) + 2.0 ** -24).all()
        assert (d == 0).double().mean() > 0.99

    x, _, q, s, _, _ = operands(17, m, n, k, bias=False, residual=False)
    near(qw.w8a16_linear(x, q, s), qw.w8a16_gemm(x, q, s))
    x, sx, q, s, _, _ = operands(18, m, n, k, a8=True, bias=False, residual=False)
    near(qw.w8a8_linear(x, sx, q, s), qw.w8a8_gemm(x, sx, q, s))


@pytest.mark.parametrize("m", [1, 6, 200])
def test_random_values(m):
    """Products that round: within the plain product's accuracy contract."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(19)
    x = torch.randn(m, 4096, generator=gen, device="cuda").half()
    q, s = qw.quantize_weights(torch.randn(1024, 4096, generator=gen, device="cuda") / 64)
    b = torch.randn(1024, generator=gen, device="cuda").half()
    want, _ = linear64(x, q, s, b, "gelu")
    got = qw.w8a16_linear(x, q, s, bias=b, activation="gelu").double()
    assert (got - want).abs().max() <= 1.13 * (2e-3 * want.abs().max() + 1e-3)


def test_large_values():
    """Sums beyond fp16's range become infinities of their sign, and the
    activations' far ends do not become NaN."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(20)
    for m, path, tile in ((1, "gemv", 0), (9, "skinny", 0), (100, "mfma", 256128), (300, "mfma", 256256)):
        x = integers(gen, (m, 256), 4, F16) * 64
        q = integers(gen, (128, 256), 127, torch.int8)
        s = scale16(gen, (128,), 64.0)
        v, _ = linear64(x, q, s)
        for act in (None, "relu", "gelu", "gelu_tanh", "silu"):
            want, off = linear64(x, q, s, act=act)
            assert_rounded(call(x, None, q, s, None, None, act, path=path, tile=tile), want, off)
        assert v.abs().max() > 1e6


def test_entry_points():
    x, sx, q, s, b, r = operands(21, 9, 64, 64, a8=True, dtype=BF16)
    want, off = linear64(x, q, s, b, "silu", False, r, sx)
    y = qw.w8a8_linear(x, sx, q, s, bias=b, activation="silu", residual=r)
    assert y.dtype == BF16
    assert_rounded(y, want, off)
    assert qw.w8a8_linear(x, sx, q, s).dtype == F16
    assert qw.w8a8_linear(x, sx, q, s, dtype=BF16).dtype == BF16
    out = torch.empty(9, 64, dtype=BF16, device="cuda")
    assert qw.w8a8_linear(x, sx, q, s, bias=b, activation="silu", residual=r, out=out) is out
    assert torch.equal(out, y)
    x, _, q, s, b, r = operands(22, 9, 64, 64, gated=True)
    want, off = linear64(x, q, s, b, "silu", True, r)
    got = qw.w8a16_linear(x, q, s, bias=b, activation="silu", gated=True, residual=r)
    assert_rounded(got, want, off)
    assert qw.w8a16_linear(x, q, s, bias=b, activation="silu", gated=True, residual=r, out=r) is r
    assert torch.equal(got, r)
    for m in (0,):
        assert qw.w8a16_linear(x[:m], q, s).shape == (0, 64)


def test_tuning_records_are_used():
    x, _, q, s, b, r = operands(23, 24, 128, 256)
    want, off = linear64(x, q, s, b, "relu", False, r)
    qw.w8a16_gemm_tune(x, q, s)
    try:
        assert_rounded(qw.w8a16_linear(x, q, s, bias=b, activation="relu", residual=r), want, off)
    finally:
        qw.tune_reset()
