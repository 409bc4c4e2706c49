"""The feed-forward half of a decoder layer (``qw_add_rms_norm``,
``qw_w8a16_linear``, ``qw_w8a8_linear``, ``qw_route_experts``,
``qw_w8a16_experts`` and ``qw_experts_combine`` of ``include/qw.h``).

    q, s, h = add_rms_norm(x, weight, residual=h, quantize=True)
    g = w8a8_linear(q, s, *gate_up, activation="silu", gated=True)
    x = w8a8_linear(*quantize_activations(g), *down, residual=h)

and with experts instead of one product for all tokens

    y, h = add_rms_norm(x, weight, residual=h)
    route = route_experts(y @ router.T, top_k)
    g = w8a16_experts(y, *gate_up, route, activation="silu", gated=True)
    d = w8a16_experts(g, *down, route, gather=False, dtype=torch.float32)
    x = experts_combine(d, route, residual=h)

As everywhere in this package, the calls check their arguments, allocate
outputs with torch and enqueue HIP kernels on the current stream; none of them
waits for the device.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import int8_weight_quantized_amd as _pkg  # (partly initialised here; its attributes are looked up when a call needs them)

from . import kv as _kv

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
SCORINGS = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 512
MAX_TOP_K = 64


class ExpertRoute(NamedTuple):
    """Where a step's tokens go.  An entry is a token and one of its experts."""
    ids: "torch.Tensor"      # int32 [tokens, top_k]: experts, -1 for none
    weights: "torch.Tensor"  # fp32 [tokens, top_k]
    offsets: "torch.Tensor"  # int32 [experts + 1]: each expert's first entry, then their number
    rows: "torch.Tensor"     # int32 [tokens * top_k]: flat index of each entry, -1 behind the last
    places: "torch.Tensor"   # int32 [tokens, top_k]: the entry of each, -1 for none


def _declare(lib):
    vp, i64, i32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
    norm = [vp, i64, vp, i64, vp, i32, i64, i64, f64, vp, i64]
    lib.qw_add_rms_norm.argtypes = norm + [vp, vp]
    lib.qw_add_rms_norm_quantize.argtypes = norm + [vp, vp, vp]
    linear = [vp, vp, vp, vp, i32, i32, vp, vp, i64, i64, i64]
    lib.qw_w8a16_linear.argtypes = linear + [vp, i64, vp]
    lib.qw_w8a16_linear_path.argtypes = linear + [i32, i32, i32, vp, i64, vp]
    linear = [vp, vp, vp, vp, vp, i32, i32, vp, i32, vp, i64, i64, i64]
    lib.qw_w8a8_linear.argtypes = linear + [vp, i64, vp]
    lib.qw_w8a8_linear_path.argtypes = linear + [i32, i32, i32, vp, i64, vp]
    for f in (lib.qw_w8a16_linear_workspace, lib.qw_w8a8_linear_workspace):
        f.argtypes = [i64, i64, i64, i32]
        f.restype = i64
    lib.qw_route_experts.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, i64, i32, f64, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.qw_route_experts_workspace.argtypes = [i64, i64, i64]
    experts = [vp, i64, i32, vp, vp, vp, i32, i32, vp, vp, i64, i64, vp, i64, i64, i64]
    lib.qw_w8a16_experts.argtypes = experts + [vp]
    lib.qw_w8a16_experts_path.argtypes = experts + [i32, i32, vp]
    lib.qw_w8a16_experts_f32.argtypes = experts + [i32, i32, vp]
    lib.qw_experts_combine.argtypes = lib.qw_experts_combine_f32.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp, i64, vp]
    for f in (lib.qw_add_rms_norm, lib.qw_add_rms_norm_quantize, lib.qw_w8a16_linear, lib.qw_w8a16_linear_path,
              lib.qw_w8a8_linear, lib.qw_w8a8_linear_path, lib.qw_route_experts, lib.qw_w8a16_experts,
              lib.qw_w8a16_experts_path, lib.qw_w8a16_experts_f32, lib.qw_experts_combine, lib.qw_experts_combine_f32):
        f.restype = i32
    lib.qw_route_experts_workspace.restype = i64


def _loaded():
    """torch, its type codes and its stream lookup (kv.py's)."""
    return _kv._torch or _kv._load_torch()


def _raise(status, where):
    if status:
        raise _pkg.QwError(status, where)


def _fits(t, dtype, shape, index):
    """Whether t is a contiguous tensor of this kind on GPU `index`: the quick
    test in front of _check, which says what is wrong."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def _rows(t, name, dtype, shape, device):
    """Check [tokens, k] activations with contiguous rows; returns the stride
    between them in elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError("%s must be [tokens, k]%s, got shape %s"
                         % (name, "" if shape is None else " = %s" % (tuple(shape),), tuple(t.shape)))
    n, k = t.shape
    s0, s1 = t.stride()
    if n <= 1:
        s0 = k
    if (s1 != 1 and k > 1) or s0 < k or s0 % 8:
        raise ValueError("%s must have contiguous rows and a stride between them that is a multiple of 8, got strides %s"
                         % (name, tuple(t.stride())))
    return s0


def _validate_norm(x, weight, residual, quantize, out, device):
    import torch
    check = _pkg._check
    sx = _rows(x, "x", None, None, device)
    code = _kv._dtype_code(x.dtype, "x")
    tokens, k = x.shape
    check(weight, "weight", x.dtype, shape=(k,), device=device)
    sr = 0 if residual is None else _rows(residual, "residual", x.dtype, (tokens, k), device)
    specs = (("q", torch.int8, (tokens, k)), ("scales", torch.float16, (tokens,))) if quantize else (("y", x.dtype, (tokens, k)),)
    h, given = None, (None,) * len(specs)
    if out is not None:
        if not isinstance(out, (tuple, list)) or len(out) != len(specs) + 1:
            raise ValueError("out must hold %d tensors (%s and h)" % (len(specs) + 1, ", ".join(s[0] for s in specs)))
        *given, h = out
        if residual is None and h is not None:
            raise ValueError("without a residual h is x itself: pass None for it")
    made = []
    for t, (name, dtype, shape) in zip(given, specs):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=device)
        else:
            check(t, name, dtype, shape=shape, device=device)
        made.append(t)
    if residual is None:
        return code, tokens, k, sx, 0, made, None, 0
    if h is None:
        return code, tokens, k, sx, sr, made, torch.empty((tokens, k), dtype=x.dtype, device=device), k
    return code, tokens, k, sx, sr, made, h, _rows(h, "h", x.dtype, (tokens, k), device)


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, quantize: bool = False, out=None):
    """h = x + residual and y = h * weight / sqrt(mean(h^2) + eps), row by row:
    x and residual fp16 or bf16 [T, K] (strided rows allowed), weight [K].
    Returns (y, h), or with ``quantize`` (q int8 [T, K], scales fp16 [T], h):
    the operands of w8a8_linear.  Without a residual h is x itself.  ``out`` is
    a tuple of the same tensors, None for those to allocate; its h may be x or
    residual (in place)."""
    torch = _loaded()
    try:
        index = x.get_device()
        dtype = x.dtype
        code = _kv._codes[dtype]
        tokens, k = x.shape
        sx, one = x.stride()
        sr = 0
        fine = (out is None and index >= 0 and one == 1 and sx >= k and sx % 8 == 0 and _fits(weight, dtype, (k,), index))
        if residual is not None:
            sr, one = residual.stride()
            fine = (fine and residual.dtype is dtype and residual.shape == x.shape and residual.get_device() == index
                    and one == 1 and sr >= k and sr % 8 == 0)
    except (AttributeError, KeyError, TypeError, ValueError):
        fine = False
    if fine:
        h = None if residual is None else torch.empty(tokens, k, dtype=dtype, device=x.device)
        sh = k
        made = ((torch.empty(tokens, k, dtype=torch.int8, device=x.device),
                 torch.empty(tokens, dtype=torch.float16, device=x.device)) if quantize
                else (torch.empty(tokens, k, dtype=dtype, device=x.device),))
    else:
        device = _pkg._require_gpu(x, "x")
        code, tokens, k, sx, sr, made, h, sh = _validate_norm(x, weight, residual, quantize, out, device)
        index = x.get_device()
    if index != _kv._current_device():
        return _pkg._on_device(index, add_rms_norm, x, weight, residual, eps, quantize, out)
    lib, stream = _pkg.library(), _kv._raw_stream(index)
    args = (x.data_ptr(), sx, _ptr(residual), sr, weight.data_ptr(), code, tokens, k, eps, _ptr(h), sh)
    if quantize:
        status = lib.qw_add_rms_norm_quantize(*args, made[0].data_ptr(), made[1].data_ptr(), stream)
    else:
        status = lib.qw_add_rms_norm(*args, made[0].data_ptr(), stream)
    if status:
        _raise(status, "qw_add_rms_norm_quantize" if quantize else "qw_add_rms_norm")
    return (*made, x if h is None else h)


# ---------------------------------------------------------------------------
# products with an epilogue
# ---------------------------------------------------------------------------

def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError("activation must be one of %s, got %r" % (sorted(a for a in ACTIVATIONS if a), name)) from None


def _workspace(need, device):
    """Scratch memory of a product whose reduction is split: (tensor or None,
    its address, its bytes).  Most take none."""
    if need <= 0:
        return None, None, 0
    t = _kv._torch.empty(need, dtype=_kv._torch.uint8, device=device)
    return t, t.data_ptr(), need


def _validate_linear(x, q, scales, bias, gated, residual, out, dtype, device, sx=None):
    import torch
    check = _pkg._check
    a8 = sx is not None
    check(x, "qx" if a8 else "x", torch.int8 if a8 else torch.float16, ndim=2, device=device)
    m, k = x.shape
    check(q, "q", torch.int8, ndim=2, device=device)
    n = q.shape[0]
    check(q, "q", torch.int8, shape=(n, k), device=device)
    check(scales, "scales", torch.float16, shape=(n,), device=device)
    if a8:
        check(sx, "sx", torch.float16, shape=(m,), device=device)
    if gated and n % 2:
        raise ValueError("a gated product needs an even number of channels, got %d" % n)
    columns = n // 2 if gated else n
    if bias is not None:
        check(bias, "bias", dtype, shape=(n,), device=device)
    if residual is not None:
        check(residual, "residual", dtype, shape=(m, columns), device=device)
    if out is None:
        out = torch.empty((m, columns), dtype=dtype, device=device)
    else:
        check(out, "out", dtype, shape=(m, columns), device=device)
    return m, n, k, out


def w8a16_linear(x, q, scales, bias=None, activation=None, gated: bool = False, residual=None, out=None):
    """act(x * dequant(q)^T + bias) + residual: x fp16 [M, K], q int8 [N, K],
    scales fp16 [N], bias fp16 [N] -> fp16 [M, N].  ``activation``: None,
    "relu", "gelu", "gelu_tanh" or "silu".  ``gated``: the weight holds a gate's
    N / 2 channels and then the other factor's, and the result [M, N / 2] is
    act(gate) * other.  residual has the result's shape, and may be ``out``."""
    torch = _loaded()
    act = _activation(activation)
    f16 = torch.float16
    try:
        index = x.get_device()
        m, k = x.shape
        n = q.shape[0]
        columns = n // 2 if gated else n
        fine = (out is None and index >= 0 and x.dtype is f16 and x.is_contiguous() and _fits(q, torch.int8, (n, k), index)
                and _fits(scales, f16, (n,), index) and not (gated and n % 2)
                and (bias is None or _fits(bias, f16, (n,), index))
                and (residual is None or _fits(residual, f16, (m, columns), index)))
    except (AttributeError, TypeError, ValueError, IndexError):
        fine = False
    if fine:
        y = torch.empty(m, columns, dtype=f16, device=x.device)
    else:
        device = _pkg._require_gpu(x, "x")
        m, n, k, y = _validate_linear(x, q, scales, bias, gated, residual, out, f16, device)
        index = x.get_device()
    if index != _kv._current_device():
        return _pkg._on_device(index, w8a16_linear, x, q, scales, bias, activation, gated, residual, out)
    lib = _pkg.library()
    _held, ws, size = _workspace(lib.qw_w8a16_linear_workspace(m, n, k, 1 if gated else 0) if m > 4 else 0, x.device)
    status = lib.qw_w8a16_linear(
        x.data_ptr(), q.data_ptr(), scales.data_ptr(), _ptr(bias), act, 1 if gated else 0, _ptr(residual), y.data_ptr(), m, n, k,
        ws, size, _kv._raw_stream(index))
    if status:
        _raise(status, "qw_w8a16_linear")
    return y


def w8a8_linear(qx, sx, q, scales, bias=None, activation=None, gated: bool = False, residual=None, dtype=None, out=None):
    """w8a16_linear for int8 activations qx [M, K] with one fp16 scale a row in
    sx [M] (add_rms_norm's or quantize_activations's).  bias, residual and the
    result are fp16 or bf16: ``dtype``, by default residual's, out's or bias's,
    else fp16."""
    torch = _loaded()
    act = _activation(activation)
    if dtype is None:
        dtype = next((t.dtype for t in (residual, out, bias) if t is not None and hasattr(t, "dtype")), torch.float16)
    f16 = torch.float16
    try:
        index = qx.get_device()
        code = _kv._codes[dtype]
        m, k = qx.shape
        n = q.shape[0]
        columns = n // 2 if gated else n
        fine = (out is None and index >= 0 and qx.dtype is torch.int8 and qx.is_contiguous() and _fits(sx, f16, (m,), index)
                and _fits(q, torch.int8, (n, k), index) and _fits(scales, f16, (n,), index) and not (gated and n % 2)
                and (bias is None or _fits(bias, dtype, (n,), index))
                and (residual is None or _fits(residual, dtype, (m, columns), index)))
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if fine:
        y = torch.empty(m, columns, dtype=dtype, device=qx.device)
    else:
        device = _pkg._require_gpu(qx, "qx")
        code = _kv._dtype_code(dtype, "dtype")
        if sx is None:
            raise TypeError("sx must be a torch.Tensor")
        m, n, k, y = _validate_linear(qx, q, scales, bias, gated, residual, out, dtype, device, sx=sx)
        index = qx.get_device()
    if index != _kv._current_device():
        return _pkg._on_device(index, w8a8_linear, qx, sx, q, scales, bias, activation, gated, residual, dtype, out)
    lib = _pkg.library()
    _held, ws, size = _workspace(lib.qw_w8a8_linear_workspace(m, n, k, 1 if gated else 0) if m > 4 else 0, qx.device)
    status = lib.qw_w8a8_linear(
        qx.data_ptr(), sx.data_ptr(), q.data_ptr(), scales.data_ptr(), _ptr(bias), act, 1 if gated else 0, _ptr(residual), code,
        y.data_ptr(), m, n, k, ws, size, _kv._raw_stream(index))
    if status:
        _raise(status, "qw_w8a8_linear")
    return y


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def _validate_route(logits, top_k, bias, groups, top_groups, device):
    import torch
    check = _pkg._check
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.float16, torch.bfloat16, torch.float32):
        raise TypeError("logits must be a float16, bfloat16 or float32 torch.Tensor")
    check(logits, "logits", logits.dtype, ndim=2, device=device)
    tokens, experts = logits.shape
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError("1 to %d experts, got %d" % (MAX_EXPERTS, experts))
    if not 1 <= top_k <= MAX_TOP_K:
        raise ValueError("top_k must be 1 to %d, got %r" % (MAX_TOP_K, top_k))
    if bias is not None:
        check(bias, "bias", torch.float32, shape=(experts,), device=device)
    if not 1 <= groups <= 64 or experts % groups:
        raise ValueError("groups must be 1 to 64 and divide the %d experts, got %r" % (experts, groups))
    if not 1 <= top_groups <= groups:
        raise ValueError("top_groups must be 1 to %d, got %r" % (groups, top_groups))
    return tokens, experts


def route_experts(logits, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                  renormalize: bool = True, scale: float = 1.0) -> ExpertRoute:
    """The top_k experts of each token by its logits (fp16, bf16 or fp32 [T, E])
    and their weights; and the entries listed expert by expert.

    Scores are a softmax or a sigmoid of the logits.  ``bias`` (fp32 [E]) is
    added to them for the choice alone, not for the weights.  With ``groups``,
    only experts of the top_groups groups of neighbours are eligible (a group's
    score: its two largest choices' sum with a bias, else its largest).
    ``renormalize`` divides a token's weights by their sum; ``scale`` multiplies
    them.  Ties go to the lowest index.  Logits of -inf or NaN are not eligible:
    a row of them is a token that goes to no expert."""
    torch = _loaded()
    if scoring not in SCORINGS:
        raise ValueError("scoring must be one of %s, got %r" % (sorted(SCORINGS), scoring))
    try:
        index = logits.get_device()
        dtype = logits.dtype
        code = 2 if dtype is torch.float32 else _kv._codes[dtype]
        tokens, experts = logits.shape
        fine = (index >= 0 and logits.is_contiguous() and 1 <= experts <= MAX_EXPERTS and 1 <= top_k <= MAX_TOP_K
                and 1 <= groups <= 64 and experts % groups == 0 and 1 <= top_groups <= groups
                and (bias is None or _fits(bias, torch.float32, (experts,), index)))
    except (AttributeError, KeyError, TypeError, ValueError):
        fine = False
    if not fine:
        device = _pkg._require_gpu(logits, "logits")
        tokens, experts = _validate_route(logits, top_k, bias, groups, top_groups, device)
        index = logits.get_device()
        code = 2 if logits.dtype is torch.float32 else _kv._codes[logits.dtype]
    if index != _kv._current_device():
        return _pkg._on_device(index, route_experts, logits, top_k, scoring, bias, groups, top_groups, renormalize, scale)
    lib = _pkg.library()
    need = lib.qw_route_experts_workspace(tokens, experts, top_k)
    if need < 0:
        raise ValueError("route_experts does not take these sizes")
    entries = tokens * top_k
    # one allocation: ids, places, weights, rows and offsets, and the workspace
    # (from 16 bytes on); a call of few tokens is bound by the host
    rest = -(experts + 1) % 4 + need // 4
    buf = torch.empty(4 * entries + experts + 1 + rest, dtype=torch.int32, device=logits.device)
    p = buf.data_ptr()
    places, weights, rows, offsets = p + 4 * entries, p + 8 * entries, p + 12 * entries, p + 16 * entries
    ws = p + 4 * buf.shape[0] - need
    status = lib.qw_route_experts(
        logits.data_ptr(), code, tokens, experts, top_k, SCORINGS[scoring], _ptr(bias), groups, top_groups,
        1 if renormalize else 0, scale, p, weights, offsets, rows, places, ws, need, _kv._raw_stream(index))
    if status:
        _raise(status, "qw_route_experts")
    ids, places, weights, rows, offsets, _ = buf.split_with_sizes((entries, entries, entries, entries, experts + 1, rest))
    shape = (tokens, top_k)
    return ExpertRoute(ids.view(shape), weights.view(torch.float32).view(shape), offsets, rows, places.view(shape))


def _check_route(route):
    if not isinstance(route, ExpertRoute):
        raise TypeError("route must be an ExpertRoute (route_experts's), got %r" % type(route).__name__)


def _validate_experts(x, q, scales, route, bias, gated, gather, out, device, dtype=None):
    import torch
    check = _pkg._check
    if dtype is None:
        dtype = torch.float16
    if dtype not in (torch.float16, torch.float32):
        raise TypeError("dtype must be torch.float16 or torch.float32, got %r" % (dtype,))
    check(x, "x", torch.float16, ndim=2, device=device)
    x_rows, k = x.shape
    _check_route(route)
    check(route.ids, "route.ids", torch.int32, ndim=2, device=device)
    tokens, top_k = route.ids.shape
    entries = tokens * top_k
    if x_rows != (tokens if gather else entries):
        raise ValueError("x must have a row for each of the %d %s, got %d"
                         % (tokens if gather else entries, "tokens" if gather else "entries", x_rows))
    check(q, "q", torch.int8, ndim=3, device=device)
    experts, n, _ = q.shape
    check(q, "q", torch.int8, shape=(experts, n, k), device=device)
    check(scales, "scales", torch.float16, shape=(experts, n), device=device)
    check(route.offsets, "route.offsets", torch.int32, shape=(experts + 1,), device=device)
    check(route.rows, "route.rows", torch.int32, shape=(entries,), device=device)
    if bias is not None:
        check(bias, "bias", torch.float16, shape=(experts, n), device=device)
    if gated and n % 2:
        raise ValueError("a gated product needs an even number of channels, got %d" % n)
    shape = (entries, n // 2 if gated else n)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    else:
        check(out, "out", dtype, shape=shape, device=device)
    return x_rows, k, top_k, entries, experts, n, out


def w8a16_experts(x, q, scales, route: ExpertRoute, bias=None, activation=None, gated: bool = False, gather: bool = True,
                  out=None, dtype=None):
    """w8a16_linear of each entry's row with its expert's weight: x fp16 [T, K]
    (a row a token), or without ``gather`` [T * top_k, K] (a row an entry, in the
    route's order), q int8 [E, N, K], scales fp16 [E, N], bias fp16 [E, N]
    -> [T * top_k, N or, gated, N / 2] in the route's order; rows behind the last
    entry are zero.  ``dtype``: torch.float16 (the default), or torch.float32 for
    entries that experts_combine adds unrounded."""
    torch = _loaded()
    act = _activation(activation)
    f16, i32 = torch.float16, torch.int32
    if dtype is None:
        dtype = f16
    try:
        index = x.get_device()
        x_rows, k = x.shape
        tokens, top_k = route.ids.shape
        entries = tokens * top_k
        experts, n, _ = q.shape
        fine = (out is None and (dtype is f16 or dtype is torch.float32) and index >= 0 and x.dtype is f16
                and x.is_contiguous() and x_rows == (tokens if gather else entries)
                and _fits(q, torch.int8, (experts, n, k), index) and _fits(scales, f16, (experts, n), index)
                and _fits(route.offsets, i32, (experts + 1,), index) and _fits(route.rows, i32, (entries,), index)
                and (bias is None or _fits(bias, f16, (experts, n), index)) and not (gated and n % 2))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if fine:
        y = torch.empty(entries, n // 2 if gated else n, dtype=dtype, device=x.device)
    else:
        device = _pkg._require_gpu(x, "x")
        x_rows, k, top_k, entries, experts, n, y = _validate_experts(x, q, scales, route, bias, gated, gather, out, device, dtype)
        index = x.get_device()
    if index != _kv._current_device():
        return _pkg._on_device(index, w8a16_experts, x, q, scales, route, bias, activation, gated, gather, out, dtype)
    lib = _pkg.library()
    args = (x.data_ptr(), x_rows, 1 if gather else 0, q.data_ptr(), scales.data_ptr(), _ptr(bias), act, 1 if gated else 0,
            route.offsets.data_ptr(), route.rows.data_ptr(), entries, top_k, y.data_ptr(), experts, n, k)
    if dtype is f16:
        status = lib.qw_w8a16_experts(*args, _kv._raw_stream(index))
    else:
        status = lib.qw_w8a16_experts_f32(*args, 0, 0, _kv._raw_stream(index))
    if status:
        _raise(status, "qw_w8a16_experts" if dtype is f16 else "qw_w8a16_experts_f32")
    return y


def _validate_combine(y, route, residual, out, device):
    import torch
    check = _pkg._check
    f32 = isinstance(y, torch.Tensor) and y.dtype == torch.float32
    check(y, "y", torch.float32 if f32 else torch.float16, ndim=2, device=device)
    n = y.shape[1]
    _check_route(route)
    check(route.places, "route.places", torch.int32, ndim=2, device=device)
    tokens, top_k = route.places.shape
    check(y, "y", y.dtype, shape=(tokens * top_k, n), device=device)
    check(route.weights, "route.weights", torch.float32, shape=(tokens, top_k), device=device)
    if residual is not None:
        check(residual, "residual", torch.float16, shape=(tokens, n), device=device)
    if out is None:
        out = torch.empty((tokens, n), dtype=torch.float16, device=device)
    else:
        check(out, "out", torch.float16, shape=(tokens, n), device=device)
    return tokens, top_k, n, out


def experts_combine(y, route: ExpertRoute, residual=None, out=None):
    """residual plus the weighted sum of each token's entries: y fp16 or fp32
    [T * top_k, N] in the route's order, residual fp16 [T, N] (may be ``out``)
    -> fp16 [T, N].  A token of no expert keeps its residual, or is zero."""
    torch = _loaded()
    f16 = torch.float16
    try:
        index = y.get_device()
        entries, n = y.shape
        tokens, top_k = route.places.shape
        fine = (out is None and index >= 0 and entries == tokens * top_k and (y.dtype is f16 or y.dtype is torch.float32)
                and y.is_contiguous()
                and _fits(route.places, torch.int32, (tokens, top_k), index)
                and _fits(route.weights, torch.float32, (tokens, top_k), index)
                and (residual is None or _fits(residual, f16, (tokens, n), index)))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if fine:
        o = torch.empty(tokens, n, dtype=f16, device=y.device)
    else:
        device = _pkg._require_gpu(y, "y")
        tokens, top_k, n, o = _validate_combine(y, route, residual, out, device)
        index = y.get_device()
    if index != _kv._current_device():
        return _pkg._on_device(index, experts_combine, y, route, residual, out)
    lib = _pkg.library()
    status = (lib.qw_experts_combine if y.dtype is f16 else lib.qw_experts_combine_f32)(
        y.data_ptr(), tokens * top_k, route.places.data_ptr(), route.weights.data_ptr(), tokens, top_k, _ptr(residual),
        o.data_ptr(), n, _kv._raw_stream(index))
    if status:
        _raise(status, "qw_experts_combine" if y.dtype is f16 else "qw_experts_combine_f32")
    return o
