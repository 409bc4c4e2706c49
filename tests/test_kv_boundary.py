"""The paged KV cache calls without a GPU: what the C ABI rejects, and what
the binding rejects before a pointer reaches it."""

import pytest

torch = pytest.importorskip("torch")
qw = pytest.importorskip("int8_weight_quantized_amd")
kv = qw.kv

META = torch.device("meta")
OK, INVALID, MISALIGNED, UNSUPPORTED, LAUNCH = (qw.QW_SUCCESS, qw.QW_ERROR_INVALID_VALUE, qw.QW_ERROR_MISALIGNED,
                                                qw.QW_ERROR_UNSUPPORTED, qw.QW_ERROR_LAUNCH)

# never dereferenced: every call is rejected on the host, or has nothing to do
P = [(i + 1) << 24 for i in range(16)]


def call(name, args, **changes):
    args = dict(args)
    args.update(changes)
    return getattr(qw.library(), name)(*args.values())


PLAN = dict(past=P[0], fresh=P[1], requests=4, table=P[2], width=8, free=P[3], n_free=5, block=64, max_tokens=9, cu=P[4],
            context=P[5], positions=P[6], slots=P[7], counts=P[8], stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(requests=-1), INVALID), (dict(width=-1), INVALID), (dict(n_free=-1), INVALID), (dict(max_tokens=-1), INVALID),
    (dict(past=0), INVALID), (dict(fresh=0), INVALID), (dict(table=0), INVALID), (dict(free=0), INVALID), (dict(cu=0), INVALID),
    (dict(context=0), INVALID), (dict(positions=0), INVALID), (dict(slots=0), INVALID), (dict(counts=0), INVALID),
    (dict(block=0), UNSUPPORTED), (dict(block=48), UNSUPPORTED), (dict(block=256), UNSUPPORTED),
    (dict(requests=8192), UNSUPPORTED), (dict(width=1 << 31), UNSUPPORTED), (dict(max_tokens=1 << 31), UNSUPPORTED),
    (dict(past=P[0] + 2), MISALIGNED), (dict(slots=P[7] + 1), MISALIGNED), (dict(counts=P[8] + 3), MISALIGNED),
    (dict(slots=P[6] + 32), INVALID),        # inside positions (9 x 4 bytes)
    (dict(cu=P[0] + 12), INVALID),           # on past's last element
    (dict(counts=P[2] + 124), INVALID),      # on the table's last element
    (dict(context=P[3]), INVALID),           # on the free list
])
def test_plan_rejects(changes, status):
    assert call("qw_kv_plan", PLAN, **changes) == status


ROPE = dict(q=P[0], q_stride=512, k=P[1], k_stride=256, dtype=0, tokens=3, hq=4, hk=2, dim=128, positions=P[2], cos=P[3],
            sin=P[4], max_position=10, rot=64, interleaved=0, qw_=P[5], kw=P[6], eps=1e-6, qo=P[7], qo_stride=512, ko=P[8],
            ko_stride=256, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dtype=2), INVALID), (dict(tokens=-1), INVALID), (dict(hq=0), INVALID), (dict(hk=0), INVALID), (dict(rot=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(qw_=0), INVALID),
    (dict(kw=0), INVALID), (dict(max_position=-1), INVALID),
    (dict(dim=96), UNSUPPORTED), (dict(dim=256), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(q_stride=516), UNSUPPORTED), (dict(ko_stride=260), UNSUPPORTED),
    (dict(q_stride=(1 << 31) + 8), UNSUPPORTED),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(qo=0), INVALID), (dict(ko=0), INVALID), (dict(positions=0), INVALID),
    (dict(cos=0), INVALID), (dict(sin=0), INVALID), (dict(q_stride=504), INVALID), (dict(ko_stride=248), INVALID),
    (dict(q=P[0] + 8), MISALIGNED), (dict(ko=P[8] + 2), MISALIGNED), (dict(cos=P[3] + 4), MISALIGNED),
    (dict(positions=P[2] + 2), MISALIGNED), (dict(qw_=P[5] + 8), MISALIGNED),
    (dict(qo=P[1]), INVALID), (dict(ko=P[0] + 1024), INVALID), (dict(qo=P[0] + 16), INVALID), (dict(ko=P[7] + 1024), INVALID),
    (dict(qo=P[3]), INVALID), (dict(ko=P[6]), INVALID), (dict(qo=P[2]), INVALID),
    (dict(qo=P[0], qo_stride=520), INVALID),                               # in place, but at another stride
    (dict(q=P[0], k=P[0] + 512, q_stride=768, k_stride=768, qo=P[0], qo_stride=768, ko=P[0] + 512, ko_stride=768), INVALID),
])
def test_norm_rope_rejects(changes, status):
    assert call("qw_qk_norm_rope", ROPE, **changes) == status


WRITE = dict(k=P[0], k_stride=256, v=P[1], v_stride=256, dtype=1, tokens=5, heads=2, dim=128, slots=P[2], kc=P[3], vc=P[4],
             ks=P[5], vs=P[6], blocks=7, block=32, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dtype=-1), INVALID), (dict(tokens=-1), INVALID), (dict(blocks=0), INVALID), (dict(heads=0), INVALID),
    (dict(kc=0), INVALID), (dict(vc=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID), (dict(k=0), INVALID),
    (dict(v=0), INVALID), (dict(slots=0), INVALID), (dict(k_stride=248), INVALID), (dict(v_stride=0), INVALID),
    (dict(dim=32), UNSUPPORTED), (dict(block=8), UNSUPPORTED), (dict(k_stride=260), UNSUPPORTED),
    (dict(blocks=1 << 31), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED), (dict(heads=65536), UNSUPPORTED),
    (dict(kc=P[3] + 8), MISALIGNED), (dict(vs=P[6] + 4), MISALIGNED), (dict(k=P[0] + 2), MISALIGNED),
    (dict(slots=P[2] + 2), MISALIGNED),
    (dict(vc=P[3] + 16), INVALID), (dict(ks=P[4] + 7 * 32 * 256 - 16), INVALID), (dict(ks=P[0] + 4 * 512 + 496), INVALID),
    (dict(vs=P[2]), INVALID),
])
def test_write_rejects(changes, status):
    assert call("qw_kv_write", WRITE, **changes) == status


READ = dict(slots=P[0], tokens=5, kc=P[1], vc=P[2], ks=P[3], vs=P[4], blocks=7, block=32, heads=2, dim=128, dtype=0, k=P[5],
            v=P[6], stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dtype=3), INVALID), (dict(tokens=-1), INVALID), (dict(blocks=0), INVALID), (dict(k=0), INVALID), (dict(slots=0), INVALID),
    (dict(dim=100), UNSUPPORTED), (dict(block=0), UNSUPPORTED), (dict(v=P[6] + 8), MISALIGNED), (dict(k=P[6] + 16), INVALID),
    (dict(v=P[1]), INVALID), (dict(k=P[0]), INVALID), (dict(k=P[4]), INVALID),
])
def test_read_rejects(changes, status):
    assert call("qw_kv_read", READ, **changes) == status


ATTN = dict(q=P[0], q_stride=512, dtype=0, tokens=6, hq=4, hk=2, dim=128, kc=P[1], vc=P[2], ks=P[3], vs=P[4], blocks=40, block=64,
            table=P[5], width=20, context=P[6], cu=P[7], requests=2, max_new=3, max_context=1280, scale=0.1, causal=1, window=0,
            out=P[8], ws=P[9], ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dtype=2), INVALID), (dict(tokens=-1), INVALID), (dict(hq=3), INVALID), (dict(hk=0), INVALID), (dict(requests=-1), INVALID),
    (dict(max_new=-1), INVALID), (dict(max_context=-1), INVALID), (dict(window=-1), INVALID), (dict(width=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(ws_bytes=-1), INVALID),
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(table=0), INVALID), (dict(context=0), INVALID), (dict(cu=0), INVALID),
    (dict(kc=0), INVALID), (dict(vs=0), INVALID), (dict(q_stride=504), INVALID), (dict(blocks=0), INVALID),
    (dict(ws=0), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(dim=80), UNSUPPORTED), (dict(block=24), UNSUPPORTED), (dict(q_stride=516), UNSUPPORTED),
    (dict(requests=65536), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED), (dict(max_new=(1 << 20) + 1), UNSUPPORTED),
    (dict(max_context=1 << 31), UNSUPPORTED), (dict(window=1 << 31), UNSUPPORTED), (dict(blocks=1 << 31), UNSUPPORTED),
    (dict(q=P[0] + 8), MISALIGNED), (dict(out=P[8] + 8), MISALIGNED), (dict(ws=P[9] + 4), MISALIGNED),
    (dict(cu=P[7] + 2), MISALIGNED), (dict(ks=P[3] + 8), MISALIGNED),
    (dict(out=P[0] + 16), INVALID), (dict(out=P[1] + 512), INVALID), (dict(ws=P[8]), INVALID), (dict(out=P[6]), INVALID),
    (dict(ws=P[5]), INVALID),
])
def test_attention_rejects(changes, status):
    assert call("qw_kv_attention", ATTN, **changes) == status


def test_nothing_to_do_is_success():
    assert call("qw_qk_norm_rope", ROPE, tokens=0) == OK
    assert call("qw_kv_write", WRITE, tokens=0) == OK
    assert call("qw_kv_read", READ, tokens=0) == OK
    for change in (dict(tokens=0), dict(requests=0), dict(max_new=0)):
        assert call("qw_kv_attention", ATTN, **change) == OK


def test_workspace_sizes():
    f = qw.library().qw_kv_attention_workspace
    assert f(64, 32, 2, 128, 64, 128, 64, 1, 8192, 0) > 0
    assert f(1, 32, 2, 128, 64, 4, 1, 1, 256, 0) == 0          # one chunk
    assert f(0, 32, 2, 128, 64, 128, 64, 1, 8192, 0) == 0
    assert f(64, 32, 3, 128, 64, 128, 64, 1, 8192, 0) == -1    # heads
    assert f(64, 32, 2, 96, 64, 128, 64, 1, 8192, 0) == -1
    # the table bounds the context
    assert f(1, 32, 2, 128, 64, 4, 1, 1, 1 << 30, 0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a process without a GPU")
def test_valid_calls_without_a_device_report_launch_errors():
    for name, args in (("qw_kv_plan", PLAN), ("qw_qk_norm_rope", ROPE), ("qw_kv_write", WRITE), ("qw_kv_read", READ),
                       ("qw_kv_attention", ATTN)):
        assert call(name, args) == LAUNCH, name
    # rotation in place on the columns of a fused tensor is no overlap
    assert call("qw_qk_norm_rope", ROPE, k=P[0] + 1024, q_stride=1024, k_stride=1024, qo=P[0], qo_stride=1024, ko=P[0] + 1024,
                ko_stride=1024) == LAUNCH


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def t(shape, dtype=torch.float16, device=META):
    return torch.empty(shape, dtype=dtype, device=device)


def cache(blocks=3, heads=2, block=16, dim=64, device=META):
    return (t((blocks, heads, block, dim), torch.int8, device), t((blocks, heads, dim, block), torch.int8, device),
            t((blocks, heads), torch.float32, device), t((blocks, heads), torch.float32, device))


def test_heads_strides():
    fused = t((5, 8 * 64))
    assert kv._heads(fused[:, :256].view(5, 4, 64), "q", META) == 512
    assert kv._heads(t((5, 4, 64)), "q", META) == 256
    assert kv._heads(t((1, 4, 64)), "q", META) == 256
    assert kv._heads(t((0, 4, 64)), "q", META) == 256
    for bad in (t((5, 4, 64)).transpose(0, 1), t((5, 4, 128))[..., ::2], t((5, 8, 64))[:, ::2], t((5, 4 * 64 + 4))[:, :256].view(5, 4, 64),
                t((5, 256)), t((5, 0, 64)), t((5, 4, 96)), t((1, 4, 64)).expand(5, 4, 64)):
        with pytest.raises(ValueError):
            kv._heads(bad, "q", META)
    with pytest.raises(TypeError):
        kv._heads([1], "q", META)


@pytest.mark.parametrize("i,bad", [
    (0, t((3, 2, 16, 64), torch.uint8)), (0, t((3, 2, 24, 64), torch.int8)), (0, t((3, 2, 16, 96), torch.int8)),
    (0, t((0, 2, 16, 64), torch.int8)), (0, t((3, 16, 64), torch.int8)), (0, t((3, 4, 16, 64), torch.int8)[:, ::2]),
    (1, t((3, 2, 16, 64), torch.int8)), (1, t((2, 2, 64, 16), torch.int8)), (2, t((3, 2), torch.float16)),
    (2, t((3, 1), torch.float32)), (3, t((3, 2), torch.float32, "cpu")), (3, None),
])
def test_cache_rejections(i, bad):
    c = list(cache())
    kv._validate_cache(*c, META)
    c[i] = bad
    with pytest.raises((ValueError, TypeError)):
        kv._validate_cache(*c, META)


def test_plan_binding_rejections():
    i = lambda *s: t(s, torch.int32)  # noqa: E731
    good = (i(4), i(4), i(4, 7), i(9), 32, 100)
    assert kv._validate_plan(*good, META) == 4
    for at, bad in ((0, i(4, 1)), (0, t((4,), torch.int64)), (1, i(5)), (2, i(5, 7)), (2, i(4)), (2, i(7, 4).t()), (3, i(3, 3)),
                    (3, t((9,), torch.int32, "cpu")), (4, 33), (5, -1)):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, TypeError)):
            kv._validate_plan(*args, META)
    n = qw.KV_PLAN_MAX_REQUESTS + 1
    with pytest.raises(ValueError):
        kv._validate_plan(i(n), i(n), i(n, 1), i(1), 16, 1, META)


def test_norm_rope_binding_rejections():
    i32, f32 = torch.int32, torch.float32
    good = dict(q=t((5, 4, 64)), k=t((5, 2, 64)), positions=t((5,), i32), cos=t((9, 16), f32), sin=t((9, 16), f32),
                q_weight=t((64,)), k_weight=t((64,)), out=None)
    kv._validate_norm_rope(*good.values(), META)
    for name, bad in (("q", t((5, 4, 64), f32)), ("k", t((5, 2, 64), torch.bfloat16)), ("k", t((4, 2, 64))), ("k", t((5, 2, 128))),
                      ("positions", t((4,), i32)), ("positions", t((5,), torch.int64)), ("cos", t((9, 12), f32)),
                      ("cos", t((9, 40), f32)), ("sin", t((8, 16), f32)), ("sin", t((9, 16))), ("q_weight", None),
                      ("k_weight", t((32,))), ("q_weight", t((64,), f32)), ("out", (t((5, 4, 64)), t((5, 4, 64)))),
                      ("out", (t((5, 4, 64)),)), ("out", (t((5, 4, 64), f32), t((5, 2, 64))))):
        args = dict(good)
        args[name] = bad
        with pytest.raises((ValueError, TypeError)):
            kv._validate_norm_rope(*args.values(), META)


def test_write_and_read_binding_rejections():
    i32 = torch.int32
    good = [t((5, 2, 64)), t((5, 2, 64)), t((5,), i32), cache()]
    kv._validate_write(*good, META)
    for at, bad in ((0, t((5, 2, 64), torch.float32)), (1, t((5, 2, 64), torch.bfloat16)), (1, t((4, 2, 64))), (1, t((5, 3, 64))),
                    (2, t((4,), i32)), (2, t((5,), torch.int64)), (3, cache(heads=3)), (3, cache(dim=128)), (0, t((5, 2, 128)))):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, TypeError)):
            kv._validate_write(*args, META)
    kv._validate_read(t((5,), i32), cache(), torch.bfloat16, META)
    for slots, dtype in ((t((5, 1), i32), torch.float16), (t((5,), torch.int64), torch.float16), (t((5,), i32), torch.float32)):
        with pytest.raises((ValueError, TypeError)):
            kv._validate_read(slots, cache(), dtype, META)


def test_attention_binding_rejections():
    i32 = torch.int32
    good = dict(q=t((6, 4, 64)), cache=cache(), table=t((2, 3), i32), context=t((2,), i32), cu=t((3,), i32), max_new=3,
                max_context=None, scale=None, window=0, out=None)
    assert kv._validate_attention(*good.values(), META)[10:12] == (48, 0.125)
    for name, bad in (("q", t((6, 4, 64), torch.float32)), ("q", t((6, 3, 64))), ("q", t((6, 4, 128))), ("table", t((6,), i32)),
                      ("table", t((2, 3), torch.int64)), ("context", t((3,), i32)), ("cu", t((2,), i32)), ("max_new", -1),
                      ("max_context", -1), ("window", -1), ("out", t((6, 4, 64), torch.bfloat16)), ("out", t((6, 4, 32))),
                      ("context", t((2,), i32, "cpu"))):
        args = dict(good)
        args[name] = bad
        with pytest.raises((ValueError, TypeError)):
            kv._validate_attention(*args.values(), META)


def test_cache_constructor():
    c = qw.kv_cache(3, 2, 64, 32, device="cpu")
    assert [tuple(x.shape) for x in c] == [(3, 2, 32, 64), (3, 2, 64, 32), (3, 2), (3, 2)]
    for bad in ((0, 2, 64, 32), (3, 0, 64, 32), (3, 2, 96, 32), (3, 2, 64, 48)):
        with pytest.raises(ValueError):
            qw.kv_cache(*bad, device="cpu")


def test_public_calls_refuse_cpu_tensors():
    cpu = "cpu"
    i = torch.zeros(2, dtype=torch.int32)
    c = cache(device=cpu)
    x = t((2, 2, 64), device=cpu)
    for f in (lambda: qw.kv_plan(i, i, i.view(2, 1), i, 16, 4), lambda: qw.qk_norm_rope(x, x, i, x, x),
              lambda: qw.kv_write(x, x, i, *c), lambda: qw.kv_read(i, *c),
              lambda: qw.kv_attention(x, *c, i.view(2, 1), i, i, 1)):
        with pytest.raises(ValueError, match="GPU"):
            f()
