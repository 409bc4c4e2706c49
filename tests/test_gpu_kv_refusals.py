"""Arguments on the GPU that the KV cache calls refuse: the quick tests in
front of the public calls must not let them through, and a refused call writes
nothing."""

import pytest

torch = pytest.importorskip("torch")
import int8_weight_quantized_amd as qw  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16, F32, I32, I64, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.int8


def t(shape, dtype=F16, device="cuda:0"):
    return torch.ones(shape, dtype=dtype, device=device)


def strided(shape, dtype=F16):
    """Of that shape, every second element of the last axis."""
    return t((*shape[:-1], 2 * shape[-1]), dtype)[..., ::2]


def cache(blocks=6, heads=2, block=16, dim=64):
    return dict(k_cache=t((blocks, heads, block, dim), I8), v_cache=t((blocks, heads, dim, block), I8),
                k_scales=t((blocks, heads), F32), v_scales=t((blocks, heads), F32))


CACHE = [("k_cache", lambda: t((6, 2, 16, 64), torch.uint8)), ("k_cache", lambda: t((6, 2, 16, 64), I8, "cpu")),
         ("k_cache", lambda: t((6, 2, 16, 64), F16)),
         ("k_cache", lambda: strided((6, 2, 16, 64), I8)), ("k_cache", lambda: t((6, 2, 24, 64), I8)),
         ("k_cache", lambda: t((6, 2, 16, 96), I8)), ("k_cache", lambda: t((6, 16, 64), I8)), ("k_cache", lambda: None),
         ("v_cache", lambda: t((6, 2, 16, 64), I8)), ("v_cache", lambda: t((5, 2, 64, 16), I8)),
         ("v_cache", lambda: t((6, 2, 64, 16), torch.uint8)), ("v_cache", lambda: t((6, 2, 64, 16), I8, "cpu")),
         ("v_cache", lambda: t((6, 2, 16, 64), I8).transpose(2, 3)),
         ("k_scales", lambda: t((6, 2), F16)), ("k_scales", lambda: t((6, 3), F32)), ("k_scales", lambda: strided((6, 2), F32)),
         ("v_scales", lambda: t((5, 2), F32)), ("v_scales", lambda: t((6, 2), torch.float64)),
         ("v_scales", lambda: t((6, 2), F32, "cpu")), ("v_scales", lambda: None)]


def made(bad):
    return bad() if callable(bad) else bad


def refuses(call, good, bad, written):
    """`call` takes `good`, and with each of `bad` in its place raises and leaves
    the tensors named in `written` as they are."""
    call(**good)
    torch.cuda.synchronize()
    for name, value in bad:
        args = {k: v.clone() if k in written else v for k, v in good.items()}
        args[name] = made(value)
        before = {k: args[k].clone() for k in written if k != name}
        with pytest.raises((ValueError, TypeError, qw.QwError)):
            call(**args)
            pytest.fail("%s was taken: %r" % (name, args[name] if not isinstance(args[name], torch.Tensor) else
                                              (args[name].shape, args[name].dtype, args[name].stride(), args[name].device)))
        torch.cuda.synchronize()
        for k, v in before.items():
            assert torch.equal(args[k], v), (name, k)


def ints(*values):
    return torch.tensor(values, dtype=I32, device="cuda:0")


def test_plan_refuses():
    good = dict(past=ints(3, 20), fresh=ints(1, 2), block_table=ints(0, -1, 1, 2).view(2, 2), free_blocks=ints(3, 4, 5),
                block_size=16, max_tokens=3)
    bad = [("past", lambda: t(2, I64)), ("past", lambda: t((2, 1), I32)), ("past", lambda: t(2, I32, "cpu")),
           ("past", lambda: strided((2,), I32)), ("past", lambda: [1, 2]), ("fresh", lambda: t(3, I32)), ("fresh", lambda: t(2, F32)),
           ("fresh", lambda: t(2, I32, "cpu")), ("fresh", lambda: strided((2,), I32)), ("block_table", lambda: t((3, 2), I32)),
           ("block_table", lambda: t(2, I32)), ("block_table", lambda: t((2, 2), I32).t()), ("block_table", lambda: t((2, 2), I64)),
           ("block_table", lambda: t((2, 2), I32, "cpu")), ("free_blocks", lambda: t((3, 1), I32)), ("free_blocks", lambda: t(3, I64)),
           ("free_blocks", lambda: strided((3,), I32)), ("free_blocks", lambda: None), ("block_size", 24), ("block_size", 0),
           ("max_tokens", -1), ("free_blocks", lambda: t(3, I32, "cpu"))]
    refuses(qw.kv_plan, good, bad, ("block_table",))


def test_norm_rope_refuses():
    good = dict(q=t((5, 4, 64)), k=t((5, 2, 64)), positions=t(5, I32), cos=t((9, 16), F32), sin=t((9, 16), F32), q_weight=t(64),
                k_weight=t(64))
    bad = [("q", lambda: t((5, 4, 64), F32)), ("q", lambda: t((5, 4, 96))), ("q", lambda: t((5, 256))), ("q", lambda: t((5, 4, 64), F16, "cpu")),
           ("q", lambda: t((4, 5, 64)).transpose(0, 1)), ("q", lambda: strided((5, 4, 64))), ("q", lambda: t((1, 4, 64)).expand(5, 4, 64)),
           ("q", lambda: t((5, 4 * 64 + 4))[:, :256].view(5, 4, 64)), ("q", lambda: t((6, 4, 64))), ("q", lambda: t((5, 0, 64))),
           ("k", lambda: t((5, 2, 64), BF16)), ("k", lambda: t((4, 2, 64))), ("k", lambda: t((5, 2, 128))),
           ("k", lambda: t((2, 5, 64)).transpose(0, 1)), ("k", lambda: t((5, 2, 64), F16, "cpu")), ("k", lambda: None),
           ("positions", lambda: t(4, I32)), ("positions", lambda: t(5, I64)), ("positions", lambda: t(5, I32, "cpu")),
           ("positions", lambda: strided((5,), I32)), ("cos", lambda: t((9, 12), F32)), ("cos", lambda: t((9, 40), F32)),
           ("cos", lambda: t((9, 16), F16)), ("cos", lambda: t((16, 9), F32).t()), ("sin", lambda: t((8, 16), F32)),
           ("sin", lambda: t((9, 16), F32, "cpu")), ("sin", lambda: t((9, 16))), ("q_weight", lambda: None), ("k_weight", lambda: None),
           ("q_weight", lambda: t(64, F32)), ("k_weight", lambda: t(32)), ("k_weight", lambda: strided((64,))),
           ("q_weight", lambda: t(64, F16, "cpu")), ("eps", -1.0), ("eps", float("nan")),
           ("out", lambda: (t((5, 4, 64)),)), ("out", lambda: (t((5, 4, 64)), t((5, 4, 64)))),
           ("out", lambda: (t((5, 4, 64), F32), t((5, 2, 64)))), ("out", lambda: (t((5, 4, 64)), t((5, 2, 64), F16, "cpu")))]
    refuses(qw.qk_norm_rope, good, bad, ())


def test_write_refuses():
    good = dict(k=t((5, 2, 64)), v=t((5, 2, 64)), slots=ints(0, 1, 2, 3, 4), **cache())
    bad = CACHE + [("k", lambda: t((5, 2, 64), F32)), ("k", lambda: t((5, 3, 64))), ("k", lambda: t((5, 2, 128))), ("k", lambda: t((4, 2, 64))),
                   ("k", lambda: t((5, 2, 64), F16, "cpu")), ("k", lambda: t((2, 5, 64)).transpose(0, 1)), ("k", lambda: None),
                   ("v", lambda: t((5, 2, 64), BF16)), ("v", lambda: t((4, 2, 64))), ("v", lambda: t((1, 2, 64)).expand(5, 2, 64)),
                   ("v", lambda: strided((5, 2, 64))), ("v", lambda: t((5, 2, 64), F16, "cpu")), ("slots", lambda: t(4, I32)),
                   ("slots", lambda: t(5, I64)), ("slots", lambda: strided((5,), I32)), ("slots", lambda: t(5, I32, "cpu"))]
    refuses(qw.kv_write, good, bad, ("k_cache", "v_cache", "k_scales", "v_scales"))
    c = cache()
    with pytest.raises(qw.QwError):   # caches that overlap
        qw.kv_write(good["k"], good["v"], good["slots"], c["k_cache"], c["k_cache"].view(6, 2, 64, 16), c["k_scales"], c["v_scales"])


def test_read_refuses():
    good = dict(slots=ints(0, 1, 95), **cache())
    bad = CACHE + [("slots", lambda: t((3, 1), I32)), ("slots", lambda: t(3, I64)), ("slots", lambda: t(3, I32, "cpu")),
                   ("slots", lambda: strided((3,), I32)), ("dtype", F32), ("dtype", I8)]
    refuses(qw.kv_read, good, bad, ())


def test_attention_refuses():
    good = dict(q=t((6, 4, 64)), **cache(), block_table=ints(0, 1, 2, 3).view(2, 2), context=ints(20, 7), cu_tokens=ints(0, 3, 6),
                max_new=3)
    bad = CACHE + [("q", lambda: t((6, 4, 64), F32)), ("q", lambda: t((6, 3, 64))), ("q", lambda: t((6, 4, 128))),
                   ("q", lambda: t((6, 4, 64), F16, "cpu")), ("q", lambda: t((4, 6, 64)).transpose(0, 1)), ("q", lambda: strided((6, 4, 64))),
                   ("q", lambda: t((1, 4, 64)).expand(6, 4, 64)), ("block_table", lambda: t(4, I32)), ("block_table", lambda: t((2, 2), I64)),
                   ("block_table", lambda: t((2, 2), I32).t()), ("block_table", lambda: t((3, 2), I32)),
                   ("block_table", lambda: t((2, 2), I32, "cpu")), ("context", lambda: t(3, I32)), ("context", lambda: t(2, I64)),
                   ("context", lambda: t(2, I32, "cpu")), ("context", lambda: strided((2,), I32)), ("cu_tokens", lambda: t(2, I32)),
                   ("cu_tokens", lambda: t(3, F32)), ("cu_tokens", lambda: t(3, I32, "cpu")), ("cu_tokens", lambda: strided((3,), I32)),
                   ("max_new", -1), ("max_context", -1), ("window", -1), ("scale", float("inf")), ("scale", float("nan")),
                   ("out", lambda: t((6, 4, 64), BF16)), ("out", lambda: t((6, 4, 32))), ("out", lambda: strided((6, 4, 64))),
                   ("out", lambda: t((6, 4, 64), F16, "cpu")), ("workspace", lambda: t(64, F32)), ("workspace", lambda: t(64, torch.uint8, "cpu"))]
    refuses(qw.kv_attention, good, bad, ())
    with pytest.raises(qw.QwError):   # in place
        qw.kv_attention(**good, out=good["q"])
    # a workspace that is too small, where one is needed
    long = dict(good, block_table=torch.zeros((2, 200), dtype=I32, device="cuda:0"), context=ints(3000, 3000))
    assert qw.kv_attention_workspace(long["q"], long["k_cache"], long["block_table"], 3) > 64
    with pytest.raises(qw.QwError):
        qw.kv_attention(**long, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda:0"))
