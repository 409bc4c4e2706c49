"""Plain 64-bit implementations of the paged KV cache operators, on the CPU,
from their formulas, and seeded inputs for them."""

from __future__ import annotations

import numpy as np

FLOOR = 2.0 ** -100


def pages(rng, contexts, block, spare=3):
    """A block table for these contexts over shuffled blocks: (table int32
    [R, W], number of blocks)."""
    need = [-(-c // block) for c in contexts]
    blocks = sum(need) + spare
    order = rng.permutation(blocks)
    width = max(1, max(need)) if need else 1
    table = np.full((len(contexts), width), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, blocks


def random_cache(rng, blocks, kv, dim, block, spread=1.0):
    """Random codes over the whole range, and positive scales over a few
    octaves (so that the blocks of a row differ)."""
    k = rng.integers(-127, 128, (blocks, kv, block, dim), dtype=np.int8)
    v = rng.integers(-127, 128, (blocks, kv, dim, block), dtype=np.int8)
    ks = (2.0 ** rng.uniform(-7 - spread, -7 + spread, (blocks, kv))).astype(np.float32)
    vs = (2.0 ** rng.uniform(-7 - spread, -7 + spread, (blocks, kv))).astype(np.float32)
    return k, v, ks, vs


def plan(past, fresh, table, free, block, max_tokens):
    table = table.copy()
    R, W = table.shape
    cu, context, positions, slots = [0], [], [], []
    used = total = 0
    for r in range(R):
        p, n = max(0, int(past[r])), max(0, int(fresh[r]))
        total += n
        n = min(n, max_tokens - cu[-1])
        cu.append(cu[-1] + n)
        context.append(min(p + n, 2 ** 31 - 1))
        held = -(-p // block)
        for pos in range(p, p + n):
            positions.append(min(pos, 2 ** 31 - 1))
            j = pos // block
            if j >= W:
                slots.append(-1)
                continue
            if pos % block == 0:  # a new block
                table[r, j] = free[used] if used < len(free) else -1
                used += 1
            b = int(table[r, j])
            s = b * block + pos % block
            slots.append(s if b >= 0 and s < 2 ** 31 else -1)
    pad = max_tokens - cu[-1]
    return dict(table=table, cu=np.array(cu), context=np.array(context, dtype=np.int64), positions=np.array(positions + [-1] * pad),
                slots=np.array(slots + [-1] * pad), counts=np.array([used, total]))


def norm_rope(x, positions, cos, sin, weight, eps, interleaved):
    """x float64 [T, H, D] -> float64, and the magnitudes that its rounding
    errors are relative to."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    out, mag = y.copy(), np.abs(y)
    rot = 2 * cos.shape[1]
    for t, p in enumerate(positions):
        if p < 0 or p >= cos.shape[0]:
            out[t] = 0.0
            continue
        c, s = cos[p].astype(np.float64), sin[p].astype(np.float64)
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = y[t][:, lo], y[t][:, hi]
        out[t][:, lo], out[t][:, hi] = a * c - b * s, b * c + a * s
        mag[t][:, lo] = np.abs(a * c) + np.abs(b * s)
        mag[t][:, hi] = np.abs(b * c) + np.abs(a * s)
    return out, mag


def runs_of(slots, block, n_slots):
    found, t = [], 0
    slots = [int(s) for s in slots]
    while t < len(slots):
        if not 0 <= slots[t] < n_slots:
            t += 1
            continue
        e = t + 1
        while e < len(slots) and slots[e] == slots[e - 1] + 1 and slots[e] % block:
            e += 1
        found.append((slots[t] // block, slots[t] % block, t, e))
        t = e
    return found


def write(x, slots, codes, scales, transposed):
    """The quantizing write of x [T, H, D] into (copies of) codes and scales.
    Scales and quotients are rounded to binary32, as the contract says."""
    codes, scales = codes.copy(), scales.copy()
    view = codes.swapaxes(2, 3) if transposed else codes
    block = view.shape[2]
    x = x.astype(np.float64)
    for b, off, lo, hi in runs_of(slots, block, view.shape[0] * block):
        for h in range(x.shape[1]):
            new = x[lo:hi, h]
            s = np.float32(np.abs(new).max() / 127.0)
            s = np.float32(0) if s < FLOOR else s
            if off and scales[b, h] >= s:
                s = scales[b, h]
            elif off and scales[b, h] > 0:
                ratio = np.float64(np.float32(np.float64(scales[b, h]) / np.float64(s)))
                view[b, h, :off] = np.rint((view[b, h, :off] * ratio).astype(np.float32))
            scales[b, h] = s
            view[b, h, off:off + hi - lo] = np.clip(np.rint((new / np.float64(s)).astype(np.float32)), -127, 127) if s > 0 else 0
    return codes, scales


def gather(slots, codes, scales, transposed):
    view = codes.swapaxes(2, 3) if transposed else codes
    block = view.shape[2]
    out = np.zeros((len(slots), view.shape[1], view.shape[3]))
    for t, s in enumerate(slots):
        if 0 <= s < view.shape[0] * block:
            out[t] = view[s // block, :, s % block].astype(np.float64) * scales[s // block].astype(np.float64)[:, None]
    return out


def attention(q, cache, table, context, cu, max_new, scale, causal=True, window=0):
    """float64 [T, Hq, D] outputs; sum_j p_j |v_j| (what weight errors are
    relative to); the largest sum_d |q_d k_d| scale of a row's keys; the
    number of keys times the largest |v|.  Rows of no request are NaN."""
    k_cache, v_cache, ks, vs = cache
    blocks, kv, block, dim = k_cache.shape
    T, heads, _ = q.shape
    group = heads // kv
    q = q.astype(np.float64)
    out = np.full(q.shape, np.nan)
    mass = np.zeros(q.shape)
    reach = np.zeros((T, heads, 1))
    tail = np.zeros((T, heads, 1))
    for r in range(table.shape[0]):
        n = min(int(cu[r + 1]) - int(cu[r]), max_new)
        ctx = min(int(context[r]), table.shape[1] * block)
        keys, vals, there = [], [], []
        for j in range(-(-ctx // block)):
            b = int(table[r, j])
            ok = 0 <= b < blocks
            b = b if ok else 0
            keys.append(k_cache[b].astype(np.float64) * ks[b].astype(np.float64)[:, None, None])
            vals.append((v_cache[b].astype(np.float64) * vs[b].astype(np.float64)[:, None, None]).swapaxes(1, 2))
            there += [ok] * block
        K = np.concatenate(keys, 1)[:, :ctx] if keys else np.zeros((kv, 0, dim))
        V = np.concatenate(vals, 1)[:, :ctx] if vals else np.zeros((kv, 0, dim))
        there = np.array(there[:ctx], bool)
        j = np.arange(ctx)
        for i in range(n):
            t, p = int(cu[r]) + i, ctx - (int(cu[r + 1]) - int(cu[r])) + i
            see = there & (j <= p if causal else True) & (j > p - window if window else True)
            for h in range(heads):
                if not see.any():
                    out[t, h] = 0.0
                    continue
                kk, vv = K[h // group][see], V[h // group][see]
                s = scale * (kk @ q[t, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                out[t, h] = w @ vv
                mass[t, h] = w @ np.abs(vv)
                reach[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
                tail[t, h] = len(kk) * np.abs(vv).max()
    return out, mass, reach, tail


def attention_rows(q, cache, table, context, cu, max_new, scale, causal=True, window=0):
    """attention() with the rows of a key head taken at once, for many rows."""
    k_cache, v_cache, ks, vs = cache
    blocks, kv, block, dim = k_cache.shape
    T, heads, _ = q.shape
    group = heads // kv
    q = q.astype(np.float64)
    out = np.full(q.shape, np.nan)
    mass = np.zeros(q.shape)
    reach = np.zeros((T, heads, 1))
    tail = np.zeros((T, heads, 1))
    for r in range(table.shape[0]):
        t0, total = int(cu[r]), int(cu[r + 1]) - int(cu[r])
        n = min(total, max_new)
        ctx = min(int(context[r]), table.shape[1] * block)
        if n <= 0:
            continue
        if ctx <= 0:
            out[t0:t0 + n] = 0.0
            continue
        ids = table[r, :-(-ctx // block)].astype(np.int64)
        ok = (ids >= 0) & (ids < blocks)
        ids = np.where(ok, ids, 0)
        there = np.repeat(ok, block)[:ctx]
        j, p = np.arange(ctx), (ctx - total + np.arange(n))[:, None]
        see = there & (j <= p if causal else True) & (j > p - window if window else True)
        see = np.repeat(np.broadcast_to(see, (n, ctx)), group, 0)
        some = see.any(1)
        for h in range(kv):
            K = (k_cache[ids, h].astype(np.float64) * ks[ids, h].astype(np.float64)[:, None, None]).reshape(-1, dim)[:ctx]
            V = (v_cache[ids, h].astype(np.float64) * vs[ids, h].astype(np.float64)[:, None, None]).swapaxes(1, 2).reshape(-1, dim)[:ctx]
            K, V = np.where(there[:, None], K, 0.0), np.where(there[:, None], V, 0.0)
            x = q[t0:t0 + n, h * group:(h + 1) * group].reshape(-1, dim)
            s = np.where(see, scale * (x @ K.T), -np.inf)
            w = np.exp(s - np.where(some, s.max(1), 0.0)[:, None])
            w /= np.where(some, w.sum(1), 1.0)[:, None]
            at = (slice(t0, t0 + n), slice(h * group, (h + 1) * group))
            out[at] = (w @ V).reshape(n, group, dim)
            mass[at] = (w @ np.abs(V)).reshape(n, group, dim)
            reach[at] = (abs(scale) * np.where(see, np.abs(x) @ np.abs(K).T, 0.0).max(1)).reshape(n, group, 1)
            tail[at] = (see.sum(1) * np.where(see, np.abs(V).max(1), 0.0).max(1)).reshape(n, group, 1)
    return out, mass, reach, tail


def attention_tolerance(out, mass, reach, tail, dim, unit):
    """One rounding of the output (`unit` of it); one fp16 rounding of each weight (2^-11 of
    it, 2^-25 where it is subnormal, relative to a largest weight of at least
    1); the scores' fp32 products and sums, dim + 8 roundings at most, as a
    relative error of the weights above and below the line."""
    return unit * np.abs(out) + (2.0 ** -11 + 2.0 ** -20 + 2 * (dim + 8) * 2.0 ** -24 * reach) * mass * (1 + unit) + 2.0 ** -25 * tail + 2.0 ** -24
