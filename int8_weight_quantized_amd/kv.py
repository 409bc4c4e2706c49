"""The paged int8 KV cache and its attention (the ``qw_kv_*`` and
``qw_qk_norm_rope`` calls of ``include/qw.h``): what a decoder layer runs
between its fused QKV GEMM and its output GEMM.

    plan = kv_plan(past, fresh, block_table, free_blocks, block_size, max_tokens)
    q, k = qk_norm_rope(q, k, plan.positions, cos, sin, q_weight, k_weight)
    kv_write(k, v, plan.slots, *cache)
    o = kv_attention(q, *cache, plan.block_table, plan.context, plan.cu_tokens, max_new)

``cache`` is the four tensors of ``kv_cache(...)``.  As everywhere in this
package, the calls check their arguments, allocate outputs with torch and
enqueue HIP kernels on the current stream; none of them waits for the device.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import int8_weight_quantized_amd as _pkg  # (partly initialised here; its attributes are looked up when a call needs them)

KV_HEAD_DIMS = (64, 128)
KV_BLOCK_SIZES = (16, 32, 64, 128)
KV_PLAN_MAX_REQUESTS = 8191
KV_ZERO_REST = 0x40000000


class KvCache(NamedTuple):
    """One layer's cache, in the order that the calls below take it."""
    k_cache: "torch.Tensor"    # int8 [blocks, kv_heads, block_size, head_dim]
    v_cache: "torch.Tensor"    # int8 [blocks, kv_heads, head_dim, block_size]
    k_scales: "torch.Tensor"   # fp32 [blocks, kv_heads]
    v_scales: "torch.Tensor"   # fp32 [blocks, kv_heads]


class KvPlan(NamedTuple):
    """A step's plan: all int32 on the device."""
    block_table: "torch.Tensor"  # [requests, table_width], updated in place
    cu_tokens: "torch.Tensor"    # [requests + 1]
    context: "torch.Tensor"      # [requests]
    positions: "torch.Tensor"    # [max_tokens]
    slots: "torch.Tensor"        # [max_tokens]
    counts: "torch.Tensor"       # [2]: blocks taken, tokens


def _declare(lib):
    vp, i64, i32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
    lib.qw_kv_plan.argtypes = [vp, vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.qw_qk_norm_rope.argtypes = [vp, i64, vp, i64, i32, i64, i64, i64, i64, vp, vp, vp, i64, i64, i32, vp, vp, f64,
                                    vp, i64, vp, i64, vp]
    lib.qw_kv_write.argtypes = [vp, i64, vp, i64, i32, i64, i64, i64, vp, vp, vp, vp, vp, i64, i64, vp]
    lib.qw_kv_read.argtypes = [vp, i64, vp, vp, vp, vp, i64, i64, i64, i64, i32, vp, vp, vp]
    lib.qw_kv_attention.argtypes = [vp, i64, i32, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, vp, i64, i64,
                                    i64, f64, i32, i64, vp, vp, i64, vp]
    for f in (lib.qw_kv_plan, lib.qw_qk_norm_rope, lib.qw_kv_write, lib.qw_kv_read, lib.qw_kv_attention):
        f.restype = i32
    lib.qw_kv_attention_workspace.argtypes = [i64] * 10
    lib.qw_kv_attention_workspace.restype = i64


# The calls below are a few microseconds of kernel each in decode, so their
# own time counts.  Each first tests its arguments with plain attribute
# reads; only where that fails do the _validate_* helpers run, which say what
# is wrong (and let pass what the quick test was too narrow for).  A kernel is
# launched on the current device, so a call whose operands are on another one
# begins again with that one current.

_torch = None
_raw_stream = None
_current_device = None


def _load_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _codes.update({torch.float16: 0, torch.bfloat16: 1})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch  # last: another thread that sees it uses the others
    return torch


_codes = {}  # torch dtype -> qw_dtype; filled with torch


def _dtype_code(dtype, name):
    _torch or _load_torch()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("%s must be torch.float16 or torch.bfloat16, got %s" % (name, dtype))
    return code


def _heads(t, name, device, heads=None, dim=None, tokens=None, dtype=None):
    """Check one [tokens, heads, head_dim] activation with contiguous heads
    and a token stride of its own; returns that stride in elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 3:
        raise ValueError("%s must be [tokens, heads, head_dim], got shape %s" % (name, tuple(t.shape)))
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) or (dim is not None and d != dim):
        raise ValueError("%s must have shape %s, got %s" % (name, (tokens, heads, dim), (n, h, d)))
    if d not in KV_HEAD_DIMS:
        raise ValueError("%s: head_dim must be one of %s, got %d" % (name, KV_HEAD_DIMS, d))
    if h == 0:
        raise ValueError("%s must have at least one head" % name)
    s0, s1, s2 = t.stride()
    if n <= 1:
        s0 = max(s0, h * d) if s0 % 8 == 0 else h * d
    if s2 != 1 or (s1 != d and h > 1) or s0 % 8 or s0 < h * d:
        raise ValueError("%s must have contiguous heads and a token stride that is a multiple of 8, got strides %s"
                         % (name, tuple(t.stride())))
    return s0


def _validate_cache(k_cache, v_cache, k_scales, v_scales, device, heads=None, dim=None):
    import torch
    check = _pkg._check
    check(k_cache, "k_cache", torch.int8, ndim=4, device=device)
    blocks, h, size, d = k_cache.shape
    if size not in KV_BLOCK_SIZES:
        raise ValueError("block_size must be one of %s, got %d" % (KV_BLOCK_SIZES, size))
    if d not in KV_HEAD_DIMS:
        raise ValueError("head_dim must be one of %s, got %d" % (KV_HEAD_DIMS, d))
    if blocks == 0 or h == 0 or (heads is not None and h != heads) or (dim is not None and d != dim):
        raise ValueError("k_cache must be [blocks, %s, block_size, %s], got %s" % (heads, dim, tuple(k_cache.shape)))
    check(v_cache, "v_cache", torch.int8, shape=(blocks, h, d, size), device=device)
    check(k_scales, "k_scales", torch.float32, shape=(blocks, h), device=device)
    check(v_scales, "v_scales", torch.float32, shape=(blocks, h), device=device)
    return blocks, h, size, d


def _validate_ints(device, **named):
    import torch
    check = _pkg._check
    for name, (t, shape) in named.items():
        check(t, name, torch.int32, shape=shape, device=device)


def _raise(status, where):
    if status:
        raise _pkg.QwError(status, where)


def kv_cache(num_blocks: int, kv_heads: int, head_dim: int, block_size: int = 64, device="cuda") -> KvCache:
    """An empty cache: zeroed codes and scales for num_blocks blocks."""
    import torch
    if head_dim not in KV_HEAD_DIMS:
        raise ValueError("head_dim must be one of %s, got %d" % (KV_HEAD_DIMS, head_dim))
    if block_size not in KV_BLOCK_SIZES:
        raise ValueError("block_size must be one of %s, got %d" % (KV_BLOCK_SIZES, block_size))
    if num_blocks < 1 or kv_heads < 1:
        raise ValueError("num_blocks and kv_heads must be positive")
    return KvCache(torch.zeros((num_blocks, kv_heads, block_size, head_dim), dtype=torch.int8, device=device),
                   torch.zeros((num_blocks, kv_heads, head_dim, block_size), dtype=torch.int8, device=device),
                   torch.zeros((num_blocks, kv_heads), dtype=torch.float32, device=device),
                   torch.zeros((num_blocks, kv_heads), dtype=torch.float32, device=device))


def _validate_plan(past, fresh, block_table, free_blocks, block_size, max_tokens, device):
    import torch
    check = _pkg._check
    check(past, "past", torch.int32, ndim=1, device=device)
    requests = past.shape[0]
    check(fresh, "fresh", torch.int32, shape=(requests,), device=device)
    check(block_table, "block_table", torch.int32, ndim=2, device=device)
    if block_table.shape[0] != requests:
        raise ValueError("block_table must have %d rows, got %d" % (requests, block_table.shape[0]))
    check(free_blocks, "free_blocks", torch.int32, ndim=1, device=device)
    if block_size not in KV_BLOCK_SIZES:
        raise ValueError("block_size must be one of %s, got %r" % (KV_BLOCK_SIZES, block_size))
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    if requests > KV_PLAN_MAX_REQUESTS:
        raise ValueError("at most %d requests, got %d" % (KV_PLAN_MAX_REQUESTS, requests))
    return requests


def kv_plan(past, fresh, block_table, free_blocks, block_size: int, max_tokens: int) -> KvPlan:
    """Block tables and slot maps of one step: request r holds past[r] tokens
    (int32 [R]) and adds fresh[r]; new blocks are taken from free_blocks
    (int32) in order and entered into block_table (int32 [R, W], in place).
    max_tokens sizes the token arrays (their padding is -1)."""
    torch = _torch or _load_torch()
    i32 = torch.int32
    try:
        index = past.get_device()
        requests, = past.shape
        rows, width = block_table.shape
        n_free, = free_blocks.shape
        fine = (index >= 0 and past.dtype is i32 and fresh.dtype is i32 and block_table.dtype is i32 and free_blocks.dtype is i32
                and fresh.shape == past.shape and rows == requests and past.is_contiguous() and fresh.is_contiguous()
                and block_table.is_contiguous() and free_blocks.is_contiguous() and fresh.get_device() == index
                and block_table.get_device() == index and free_blocks.get_device() == index and block_size in KV_BLOCK_SIZES
                and max_tokens >= 0 and requests <= KV_PLAN_MAX_REQUESTS)
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        device = _pkg._require_gpu(past, "past")
        requests = _validate_plan(past, fresh, block_table, free_blocks, block_size, max_tokens, device)
        index, width, n_free = past.get_device(), block_table.shape[1], free_blocks.shape[0]
    if index != _current_device():
        return _pkg._on_device(index, kv_plan, past, fresh, block_table, free_blocks, block_size, max_tokens)
    # one allocation for the five arrays
    buf = torch.empty(2 * requests + 3 + 2 * max_tokens, dtype=i32, device=past.device)
    cu, context, counts, positions, slots = buf.split_with_sizes((requests + 1, requests, 2, max_tokens, max_tokens))
    p = buf.data_ptr()
    p_ctx = p + 4 * (requests + 1)
    p_counts = p_ctx + 4 * requests
    p_pos = p_counts + 8
    status = _pkg.library().qw_kv_plan(
        past.data_ptr(), fresh.data_ptr(), requests, block_table.data_ptr(), width, free_blocks.data_ptr(), n_free, block_size,
        max_tokens, p, p_ctx, p_pos, p_pos + 4 * max_tokens, p_counts, _raw_stream(index))
    if status:
        _raise(status, "qw_kv_plan")
    return KvPlan(block_table, cu, context, positions, slots, counts)


def _validate_norm_rope(q, k, positions, cos, sin, q_weight, k_weight, out, device):
    import torch
    check = _pkg._check
    code = _dtype_code(q.dtype, "q")
    sq = _heads(q, "q", device)
    tokens, hq, dim = q.shape
    sk = _heads(k, "k", device, dim=dim, tokens=tokens, dtype=q.dtype)
    hk = k.shape[1]
    check(positions, "positions", torch.int32, shape=(tokens,), device=device)
    check(cos, "cos", torch.float32, ndim=2, device=device)
    check(sin, "sin", torch.float32, shape=tuple(cos.shape), device=device)
    rot = 2 * cos.shape[1]
    if rot > dim or rot % 16:
        raise ValueError("cos and sin must have rot_dim / 2 columns with rot_dim a multiple of 16 up to %d, got %d" % (dim, rot))
    if (q_weight is None) != (k_weight is None):
        raise ValueError("pass both q_weight and k_weight, or neither")
    if q_weight is not None:
        check(q_weight, "q_weight", q.dtype, shape=(dim,), device=device)
        check(k_weight, "k_weight", q.dtype, shape=(dim,), device=device)
    if out is None:
        qo = torch.empty((tokens, hq, dim), dtype=q.dtype, device=device)
        ko = torch.empty((tokens, hk, dim), dtype=q.dtype, device=device)
        return code, tokens, hq, hk, dim, rot, sq, sk, qo, hq * dim, ko, hk * dim
    qo, ko = out
    sqo = _heads(qo, "out[0]", device, heads=hq, dim=dim, tokens=tokens, dtype=q.dtype)
    sko = _heads(ko, "out[1]", device, heads=hk, dim=dim, tokens=tokens, dtype=q.dtype)
    return code, tokens, hq, hk, dim, rot, sq, sk, qo, sqo, ko, sko


def qk_norm_rope(q, k, positions, cos, sin, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 out=None):
    """RMS norm of every query and key head (skipped without weights) and the
    rotation by position, in one pass: q [T, Hq, D], k [T, Hk, D] fp16 or
    bf16 (strided token views allowed), positions int32 [T], cos and sin fp32
    [P, rot_dim / 2].  ``interleaved`` rotates pairs (2 i, 2 i + 1), else
    (i, i + rot_dim / 2).  Returns (q, k); ``out=(q, k)`` rotates in place."""
    torch = _torch or _load_torch()
    try:
        index = q.get_device()
        dtype = q.dtype
        code = _codes[dtype]
        tokens, hq, dim = q.shape
        hk = k.shape[1]
        span, half = cos.shape
        rot = 2 * half
        sq, sk = q.stride(), k.stride()
        fine = (out is None and index >= 0 and sq[0] >= hq * dim and sk[0] >= hk * dim and dim in KV_HEAD_DIMS and k.shape == (tokens, hk, dim)
                and k.dtype is dtype and sq[2] == 1 and sk[2] == 1 and sq[1] == dim and sk[1] == dim and sq[0] % 8 == 0
                and sk[0] % 8 == 0 and hq > 0 and hk > 0 and k.get_device() == index
                and positions.dtype is torch.int32 and positions.shape == (tokens,) and positions.is_contiguous()
                and positions.get_device() == index and cos.dtype is torch.float32 and sin.dtype is torch.float32
                and sin.shape == cos.shape and cos.is_contiguous() and sin.is_contiguous() and cos.get_device() == index
                and sin.get_device() == index and rot <= dim and rot % 16 == 0)
        if fine and q_weight is not None:
            fine = (q_weight.dtype is dtype and k_weight.dtype is dtype and q_weight.shape == (dim,) and k_weight.shape == (dim,)
                    and q_weight.is_contiguous() and k_weight.is_contiguous() and q_weight.get_device() == index
                    and k_weight.get_device() == index)
        elif fine:
            fine = k_weight is None
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if fine:
        sq, sk, sqo, sko = sq[0], sk[0], hq * dim, hk * dim
        # (strided views and heads in order: new tensors of their kind are contiguous)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
    else:
        device = _pkg._require_gpu(q, "q")
        code, tokens, hq, hk, dim, rot, sq, sk, qo, sqo, ko, sko = _validate_norm_rope(
            q, k, positions, cos, sin, q_weight, k_weight, out, device)
        index, span = q.get_device(), cos.shape[0]
    if index != _current_device():
        return _pkg._on_device(index, qk_norm_rope, q, k, positions, cos, sin, q_weight, k_weight, eps, interleaved, out)
    status = _pkg.library().qw_qk_norm_rope(
        q.data_ptr(), sq, k.data_ptr(), sk, code, tokens, hq, hk, dim, positions.data_ptr(), cos.data_ptr(), sin.data_ptr(),
        span, rot, 1 if interleaved else 0, None if q_weight is None else q_weight.data_ptr(),
        None if k_weight is None else k_weight.data_ptr(), eps, qo.data_ptr(), sqo, ko.data_ptr(), sko, _raw_stream(index))
    if status:
        _raise(status, "qw_qk_norm_rope")
    return qo, ko


def _cache_fits(k_cache, v_cache, k_scales, v_scales, index):
    """Whether the four tensors are a cache on device `index` (the quick test
    of _validate_cache)."""
    torch = _torch
    blocks, heads, size, dim = k_cache.shape
    return (dim in KV_HEAD_DIMS and size in KV_BLOCK_SIZES and blocks > 0 and heads > 0
            and k_cache.dtype is torch.int8 and v_cache.dtype is torch.int8 and k_scales.dtype is torch.float32
            and v_scales.dtype is torch.float32 and v_cache.shape == (blocks, heads, dim, size)
            and k_scales.shape == (blocks, heads) and v_scales.shape == (blocks, heads) and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous()
            and k_cache.get_device() == index and v_cache.get_device() == index and k_scales.get_device() == index
            and v_scales.get_device() == index)


def _validate_write(k, v, slots, cache, device):
    import torch
    code = _dtype_code(k.dtype, "k")
    sk = _heads(k, "k", device)
    tokens, heads, dim = k.shape
    sv = _heads(v, "v", device, heads=heads, dim=dim, tokens=tokens, dtype=k.dtype)
    blocks, _, size, _ = _validate_cache(*cache, device, heads=heads, dim=dim)
    _pkg._check(slots, "slots", torch.int32, shape=(tokens,), device=device)
    return code, tokens, heads, dim, sk, sv, blocks, size


def kv_write(k, v, slots, k_cache, v_cache, k_scales, v_scales) -> None:
    """Quantize new keys and values (fp16 or bf16 [T, H, D], strided token
    views allowed) into the cache at slots (int32 [T]; -1 skips a token).
    The tokens of a block follow each other in one call, as kv_plan numbers
    them; a block's scale grows to the largest value it holds."""
    torch = _torch or _load_torch()
    try:
        index = k.get_device()
        dtype = k.dtype
        code = _codes[dtype]
        tokens, heads, dim = k.shape
        blocks, cache_heads, size, cache_dim = k_cache.shape
        sk, sv = k.stride(), v.stride()
        fine = (index >= 0 and sk[0] >= heads * dim and sv[0] >= heads * dim and v.shape == k.shape and v.dtype is dtype and sk[2] == 1 and sv[2] == 1
                and sk[1] == dim and sv[1] == dim and sk[0] % 8 == 0 and sv[0] % 8 == 0 and v.get_device() == index
                and slots.dtype is torch.int32 and slots.shape == (tokens,) and slots.is_contiguous()
                and slots.get_device() == index and cache_heads == heads and cache_dim == dim
                and _cache_fits(k_cache, v_cache, k_scales, v_scales, index))
        sk, sv = sk[0], sv[0]
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        device = _pkg._require_gpu(k, "k")
        code, tokens, heads, dim, sk, sv, blocks, size = _validate_write(k, v, slots, (k_cache, v_cache, k_scales, v_scales), device)
        index = k.get_device()
    if index != _current_device():
        return _pkg._on_device(index, kv_write, k, v, slots, k_cache, v_cache, k_scales, v_scales)
    status = _pkg.library().qw_kv_write(
        k.data_ptr(), sk, v.data_ptr(), sv, code, tokens, heads, dim, slots.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), blocks, size, _raw_stream(index))
    if status:
        _raise(status, "qw_kv_write")


def _validate_read(slots, cache, dtype, device):
    import torch
    code = _dtype_code(dtype, "dtype")
    _pkg._check(slots, "slots", torch.int32, ndim=1, device=device)
    blocks, heads, size, dim = _validate_cache(*cache, device)
    return code, slots.shape[0], blocks, heads, size, dim


def kv_read(slots, k_cache, v_cache, k_scales, v_scales, dtype=None):
    """The keys and values that slots (int32 [T]) of the cache stand for, in
    fp16 (or the given 16-bit dtype): (k, v), each [T, H, D]; zeros for -1."""
    torch = _torch or _load_torch()
    dtype = torch.float16 if dtype is None else dtype
    try:
        index = slots.get_device()
        code = _codes[dtype]
        tokens, = slots.shape
        blocks, heads, size, dim = k_cache.shape
        fine = (index >= 0 and slots.dtype is torch.int32 and slots.is_contiguous()
                and _cache_fits(k_cache, v_cache, k_scales, v_scales, index))
    except (AttributeError, KeyError, TypeError, ValueError):
        fine = False
    if not fine:
        device = _pkg._require_gpu(slots, "slots")
        code, tokens, blocks, heads, size, dim = _validate_read(slots, (k_cache, v_cache, k_scales, v_scales), dtype, device)
        index = slots.get_device()
    if index != _current_device():
        return _pkg._on_device(index, kv_read, slots, k_cache, v_cache, k_scales, v_scales, dtype)
    k = torch.empty((tokens, heads, dim), dtype=dtype, device=slots.device)
    v = torch.empty_like(k)
    status = _pkg.library().qw_kv_read(
        slots.data_ptr(), tokens, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), blocks,
        size, heads, dim, code, k.data_ptr(), v.data_ptr(), _raw_stream(index))
    if status:
        _raise(status, "qw_kv_read")
    return k, v


def _validate_attention(q, cache, block_table, context, cu_tokens, max_new, max_context, scale, window, out, device):
    import torch
    check = _pkg._check
    code = _dtype_code(q.dtype, "q")
    sq = _heads(q, "q", device)
    tokens, heads, dim = q.shape
    blocks, kv_heads, size, _ = _validate_cache(*cache, device, dim=dim)
    if heads % kv_heads:
        raise ValueError("%d query heads are not a multiple of %d key heads" % (heads, kv_heads))
    check(block_table, "block_table", torch.int32, ndim=2, device=device)
    requests, width = block_table.shape
    check(context, "context", torch.int32, shape=(requests,), device=device)
    check(cu_tokens, "cu_tokens", torch.int32, shape=(requests + 1,), device=device)
    if max_new < 0 or window < 0:
        raise ValueError("max_new and window must not be negative")
    if max_context is None:
        max_context = width * size
    elif max_context < 0:
        raise ValueError("max_context must not be negative")
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=device)
    else:
        check(out, "out", q.dtype, shape=(tokens, heads, dim), device=device)
    return code, tokens, heads, dim, sq, blocks, kv_heads, size, requests, width, max_context, scale, out


def kv_attention_workspace(q, k_cache, block_table, max_new: int, max_context=None, window: int = 0) -> int:
    """Workspace bytes that kv_attention uses for these operands."""
    tokens, heads, dim = q.shape
    requests, width = block_table.shape
    size = k_cache.shape[2]
    n = int(_pkg._on_device(
        q.get_device(), _pkg.library().qw_kv_attention_workspace, tokens, heads, k_cache.shape[1], dim, size, width, requests,
        max_new, width * size if max_context is None else max_context, window))
    if n < 0:
        raise ValueError("kv_attention does not take these sizes")
    return n


def kv_attention(q, k_cache, v_cache, k_scales, v_scales, block_table, context, cu_tokens, max_new: int, max_context=None,
                 scale=None, causal: bool = True, window: int = 0, out=None, workspace=None):
    """Attention of the new tokens' queries over the cache: q fp16 or bf16
    [T, Hq, D] (strided token views allowed), block_table int32 [R, W],
    context int32 [R] (cached tokens, the new ones among them), cu_tokens
    int32 [R + 1] (kv_plan's).  max_new is at least the most new tokens of a
    request, max_context at least the longest context (default: what the
    table holds); both are host numbers that size the launch.  window > 0
    lets a query see that many keys, its own the last.  Rows that see
    nothing are zero.  Rows of no request (padding behind the last one's tokens)
    are zero too, or keep what a given ``out`` holds there.  ``workspace`` (uint8, kv_attention_workspace bytes) is
    allocated when not given.  Returns [T, Hq, D]."""
    torch = _torch or _load_torch()
    try:
        index = q.get_device()
        dtype = q.dtype
        code = _codes[dtype]
        tokens, heads, dim = q.shape
        blocks, kv_heads, size, cache_dim = k_cache.shape
        requests, width = block_table.shape
        sq = q.stride()
        i32 = torch.int32
        fine = (out is None and index >= 0 and tokens > 0 and sq[2] == 1 and sq[1] == dim and sq[0] % 8 == 0
                and sq[0] >= heads * dim and cache_dim == dim and heads % kv_heads == 0 and block_table.dtype is i32
                and context.dtype is i32 and cu_tokens.dtype is i32 and context.shape == (requests,)
                and cu_tokens.shape == (requests + 1,) and block_table.is_contiguous() and context.is_contiguous()
                and cu_tokens.is_contiguous() and block_table.get_device() == index and context.get_device() == index
                and cu_tokens.get_device() == index and max_new >= 0 and window >= 0
                and _cache_fits(k_cache, v_cache, k_scales, v_scales, index))
        sq = sq[0]
        if max_context is None:
            max_context = width * size
        fine = fine and max_context >= 0
    except (AttributeError, KeyError, TypeError, ValueError, IndexError, ZeroDivisionError):
        fine = False
    mask, given = 1 if causal else 0, out
    if out is None:
        mask |= KV_ZERO_REST  # an output allocated here holds nothing to keep
    if fine:
        if scale is None:
            scale = 1.0 / math.sqrt(dim)
        out = torch.empty_like(q)  # (contiguous, as in qk_norm_rope)
    else:
        device = _pkg._require_gpu(q, "q")
        code, tokens, heads, dim, sq, blocks, kv_heads, size, requests, width, max_context, scale, out = _validate_attention(
            q, (k_cache, v_cache, k_scales, v_scales), block_table, context, cu_tokens, max_new, max_context, scale, window, out,
            device)
        index = q.get_device()
    if index != _current_device():
        return _pkg._on_device(index, kv_attention, q, k_cache, v_cache, k_scales, v_scales, block_table, context, cu_tokens,
                               max_new, max_context, scale, causal, window, given, workspace)
    if mask & KV_ZERO_REST and (requests == 0 or max_new == 0):
        return out.zero_()
    lib = _pkg.library()
    if workspace is None:
        need = lib.qw_kv_attention_workspace(tokens, heads, kv_heads, dim, size, width, requests, max_new, max_context, window)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _pkg._check(workspace, "workspace", torch.uint8, ndim=1, device=q.device)
        need = workspace.numel()
    status = lib.qw_kv_attention(
        q.data_ptr(), sq, code, tokens, heads, kv_heads, dim, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
        v_scales.data_ptr(), blocks, size, block_table.data_ptr(), width, context.data_ptr(), cu_tokens.data_ptr(), requests,
        max_new, max_context, scale, mask, window, out.data_ptr(),
        None if workspace is None else workspace.data_ptr(), need if need > 0 else 0, _raw_stream(index))
    if status:
        _raise(status, "qw_kv_attention")
    return out
