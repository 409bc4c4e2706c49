"""The serving operators around an int8 paged KV cache, case by case: the plan of a step (block tables, slot map), the
per-head norm and rotation of queries and keys, the quantizing write into the cache (and the read back), and attention
over it.

``own`` false: each operator in elementary torch operations, in fp32, rounded once.  ``own`` true: the calls a user makes of
``int8_weight_quantized_amd``.  ``exact`` gives the same outputs from the definitions in 64 bits.

The cache of one layer is four tensors: ``k_cache`` int8 [blocks, kv_heads, block_size, head_dim], ``v_cache`` int8
[blocks, kv_heads, head_dim, block_size], and ``k_scales``, ``v_scales`` fp32 [blocks, kv_heads]; a value is its code
times the scale of its block and head.  Token ``p`` of request ``r`` sits in slot ``block_table[r][p // block_size] *
block_size + p % block_size``.
"""

import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
TINY = 2.0 ** -100  # a block whose scale would lie below holds zeros


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    """heads/kv_heads/dim 32/2/128 is the layer behind the benchmark's fused QKV projection of 4608 channels; 32/8/128
    and 16/16/64 are the generic grouped and ungrouped layers."""
    return [
        # the scheduler's step for 64 requests that each decode one token
        plan_case("plan_decode", requests=64, new=1, past=2048, block=64),
        # a step that admits prompts beside running requests, in small blocks
        plan_case("plan_mixed", requests=512, new=256, past=8192, block=16),
        # one decode step of eight requests: launch latency
        rope_case("rope_decode", tokens=8, heads=32, kv=2, dim=128, rot=64, pairs=True, dtype="f16"),
        # a prompt batch: every query and key head of 16384 tokens
        rope_case("rope_prompt", tokens=16384, heads=32, kv=8, dim=128, rot=128, pairs=False, dtype="bf16"),
        # one token into each of 64 partly filled blocks
        write_case("write_decode", requests=64, new=1, kv=2, dim=128, block=64, dtype="f16"),
        # ragged prompts into fresh and partly filled blocks
        write_case("write_prompt", requests=13, new=2048, kv=8, dim=128, block=64, dtype="bf16"),
        # the first tokens of one conversation: launch latency
        attn_case("attn_decode_one", requests=1, new=1, past=332, heads=32, kv=2, dim=128, block=64, dtype="f16"),
        # a ragged decode batch, an idle request among it
        attn_case("attn_decode_batch", requests=64, new=1, past=8191, heads=32, kv=2, dim=128, block=64, dtype="f16"),
        # ungrouped heads in small blocks: one query row for each head's keys
        attn_case("attn_decode_ungrouped", requests=48, new=1, past=2047, heads=16, kv=16, dim=64, block=16, dtype="bf16"),
        # drafted tokens checked against two very long contexts
        attn_case("attn_draft_long", requests=2, new=5, past=131067, heads=32, kv=8, dim=128, block=32, dtype="bf16"),
        # ragged prompts, nothing cached before them
        attn_case("attn_prompt", requests=3, new=4096, past=0, heads=32, kv=2, dim=128, block=64, dtype="f16"),
        # a chunk of each of eight long prompts under a sliding window
        attn_case("attn_chunk_window", requests=8, new=512, past=15872, heads=16, kv=16, dim=64, block=128, dtype="bf16",
                  window=4096),
    ]


def plan_case(name, requests, new, past, block):
    return named(name, {"op": "plan", "requests": requests, "new": new, "past": past, "block": block})


def rope_case(name, tokens, heads, kv, dim, rot, pairs, dtype):
    return named(name, {"op": "rope", "tokens": tokens, "heads": heads, "kv": kv, "dim": dim, "rot": rot, "pairs": pairs,
                        "dtype": dtype})


def write_case(name, requests, new, kv, dim, block, dtype):
    return named(name, {"op": "write", "requests": requests, "new": new, "kv": kv, "dim": dim, "block": block, "dtype": dtype})


def attn_case(name, requests, new, past, heads, kv, dim, block, dtype, window=0):
    return named(name, {"op": "attn", "requests": requests, "new": new, "past": past, "heads": heads, "kv": kv, "dim": dim,
                        "block": block, "dtype": dtype, "window": window})


def named(name, case):
    return dict({"name": name}, **case) if name else case


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("plan", "rope", "write", "attn", "attn", "attn"))
    heads, kv, dim = rng.choice(((32, 2, 128), (32, 8, 128), (16, 16, 64), (16, 4, 64), (24, 3, 128), (28, 4, 128), (12, 12, 64)))
    block = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    if op == "plan":
        return plan_case(None, log(1, 512), log(1, 256), log(1, 8192), block)
    if op == "rope":
        return rope_case(None, log(1, 16384), heads, kv, dim, rng.choice((dim, dim // 2)), rng.random() < 0.5, dtype)
    if op == "write":
        requests = log(1, 64)
        return write_case(None, requests, log(1, 24576 // requests), kv, dim, block, dtype)
    window = rng.choice((0, 0, 0, 333, 1024))
    form = rng.choice(("decode", "draft", "prompt", "chunk"))
    if form == "decode":
        requests = log(1, 64)
        return attn_case(None, requests, 1, log(1, min(65536, 6000 * 64 // requests)), heads, kv, dim, block, dtype, window)
    if form == "draft":
        requests = log(1, 16)
        return attn_case(None, requests, rng.randint(2, 8), log(16, min(65536, 200000 // requests)), heads, kv, dim, block, dtype,
                         window)
    if form == "prompt":
        requests = log(1, 8)
        return attn_case(None, requests, log(9, int(4096 / math.sqrt(requests))), 0, heads, kv, dim, block, dtype, window)
    requests = log(1, 6)
    new = log(16, 512)
    return attn_case(None, requests, new, log(512, min(32768, 15872 * 512 // new)), heads, kv, dim, block, dtype, window)


def spread(count, most, least=0):
    """`count` lengths between least and most, the longest first, evenly uneven: the same for every seed."""
    return [most - int((most - least) * ((0.6180339887 * i) % 1.0)) for i in range(count)]


def lengths(case):
    """(tokens cached before the step, new tokens) of each request."""
    n = case["requests"]
    if case["op"] == "attn" and case["past"] == 0:  # prompts
        new = spread(n, case["new"], max(1, case["new"] // 8))
    elif case["new"] < 9:  # decode, drafts
        new = [case["new"]] * n
    else:
        new = spread(n, case["new"], 1)
    if case["op"] == "write":  # what is cached before ends anywhere in a block, or at its edge
        past = [(7 * i + 5) * case["block"] // 11 for i in range(n)]
    else:
        past = spread(n, case["past"], case["past"] // 16)
    if case["op"] == "plan" and n >= 8:
        new[n // 2] = 0  # a request that waits
    return past, new


def idle(case):
    """In a batch of decodes the last place is empty: it has a query row, and no token to attend to."""
    return case["op"] == "attn" and case["new"] == 1 and case["requests"] >= 8


def work(case):
    if case["op"] == "rope":
        rows = case["tokens"] * (case["heads"] + case["kv"])
        return {"bytes": 2.0 * 2 * rows * case["dim"] + case["tokens"] * 4.0 * (1 + case["rot"]), "flops": 8.0 * rows * case["dim"]}
    past, new = lengths(case)
    T = sum(new)
    if case["op"] == "plan":
        B = case["block"]
        taken = sum(-(-(p + n) // B) - -(-p // B) for p, n in zip(past, new))
        held = sum(1 for p, n in zip(past, new) if p % B and n)  # the table entry of a partly filled block
        return {"bytes": 4.0 * (4 * len(past) + 1 + 2 + 2 * T + 2 * taken + held), "flops": 4.0 * T}
    if case["op"] == "write":
        live = sum(n + p % case["block"] for p, n in zip(past, new))
        row = 2.0 * case["kv"] * case["dim"]
        # 16-bit rows in and codes out; the touched blocks' codes in and 16-bit rows out; scales and slots
        blocks = sum(-(-(p % case["block"] + n) // case["block"]) for p, n in zip(past, new))
        return {"bytes": T * row * 3 + live * row * 3 + 4.0 * (T + live + 4 * blocks * case["kv"]), "flops": 4.0 * (T + live) * row}
    read = pairs = 0
    for r, (p, n) in enumerate(zip(past, new)):
        if idle(case) and r == case["requests"] - 1:
            continue
        w = case["window"] or p + n
        read += min(p + n, w + n - 1)
        full = max(0, min(n, p + n - w + 1))  # rows that see the whole window
        pairs += full * w + sum(range(p + 1, p + n - full + 1))
    rows = 2.0 * T * case["heads"] * case["dim"]
    return {"bytes": read * case["kv"] * (2.0 * case["dim"] + 8.0 / case["block"]) + 2 * rows,
            "flops": 4.0 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def channels(gen, kv, dim):
    """Keys have a few channels much larger than the rest; the gain of each."""
    gain = 0.5 + torch.rand(kv, dim, generator=gen, device=DEV)
    gain[:, torch.randint(0, dim, (2,), generator=gen, device=DEV)] *= 8.0
    return gain


def cache_of(gen, blocks, case, empty=False):
    """A cache that holds normal keys (with large channels) and values, quantized block by block."""
    kv, dim, B = case["kv"], case["dim"], case["block"]
    made = []
    for shape, gain in (((blocks, kv, B, dim), channels(gen, kv, dim)[:, None, :]), ((blocks, kv, dim, B), 1.0)):
        x = normal(gen, *shape) * gain
        s = x.abs().amax(dim=(2, 3)) / 127.0
        made.append((torch.round(x / s[:, :, None, None]).clamp(-127, 127).to(torch.int8), s))
    (k, ks), (v, vs) = made
    return k, v, ks, vs


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = random.Random(seed)
    dtype = TYPES.get(case.get("dtype"))
    s = dict(case)

    if case["op"] == "rope":
        T, hq, kv, dim, rot = (case[n] for n in ("tokens", "heads", "kv", "dim", "rot"))
        s["positions"] = torch.randint(0, 8192, (T,), generator=gen, device=DEV, dtype=torch.int32)
        angle = torch.arange(8192, device=DEV).float()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=DEV).float() / rot)
        s["cos"], s["sin"] = angle.cos().contiguous(), angle.sin().contiguous()
        qkv = normal(gen, T, (hq + 2 * kv) * dim).to(dtype)  # the fused projection's output: q, k and v side by side
        s["q"] = qkv[:, :hq * dim].view(T, hq, dim)
        s["k"] = qkv[:, hq * dim:(hq + kv) * dim].view(T, kv, dim)
        s["q_weight"] = (1.0 + 0.2 * normal(gen, dim)).to(dtype)
        s["k_weight"] = (1.0 + 0.2 * normal(gen, dim)).to(dtype)
        return s

    past, new = lengths(case)
    if idle(case):
        past[-1] = -new[-1]
    at = list(zip(past, new))
    B = case["block"]
    if case["op"] == "write":
        rnd.shuffle(at)
    else:
        at = at[:1] + rnd.sample(at[1:], len(at) - 1)  # requests come in any order
    past, new = [p for p, _ in at], [n for _, n in at]
    context = [p + n for p, n in at]
    first = [0]
    for n in new:
        first.append(first[-1] + n)
    wide = max(1, max(-(-c // B) for c in context))
    held = [-(-(p if case["op"] == "plan" else c) // B) for p, c in zip(past, context)]
    blocks = sum(-(-c // B) for c in context) + 7
    order = list(range(blocks))
    rnd.shuffle(order)
    table, used = [], 0
    for h in held:
        table.append(order[used:used + h] + [-1] * (wide - h))
        used += h

    if case["op"] == "plan":
        s.update(past=ints(past), new=ints(new), table=ints(table), free=ints(order[used:]), total=first[-1])
        return s

    T, kv, dim = first[-1], case["kv"], case["dim"]
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = cache_of(gen, blocks, case)
    if case["op"] == "write":
        def slots(r, lo, hi):
            return [table[r][p // B] * B + p % B for p in range(lo, hi)]
        s["slots"] = ints([x for r, (p, n) in enumerate(at) for x in slots(r, p, p + n)])
        # every live token of the blocks that the write touches
        s["live"] = ints([x for r, (p, n) in enumerate(at) for x in slots(r, p - p % B, p + n)])
        s["k"] = (normal(gen, T, kv, dim) * channels(gen, kv, dim)).to(dtype)
        s["v"] = normal(gen, T, kv, dim).to(dtype)
        return s

    s.update(table=ints(table), context=ints(context), cu=ints(first), max_new=max(new), max_context=max(context))
    s["q"] = normal(gen, T, case["heads"], dim).to(dtype)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def own_plan(s):
    import int8_weight_quantized_amd as qw
    p = qw.kv_plan(s["past"], s["new"], s["table"], s["free"], s["block"], s["total"])
    return {"table": p.block_table, "cu": p.cu_tokens, "context": p.context, "positions": p.positions, "slots": p.slots,
            "counts": p.counts}


def own_rope(s):
    import int8_weight_quantized_amd as qw
    q, k = qw.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos"], s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                           eps=1e-6, interleaved=s["pairs"])
    return {"q": q, "k": k}


def own_write(s):
    import int8_weight_quantized_amd as qw
    cache = (s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
    qw.kv_write(s["k"], s["v"], s["slots"], *cache)
    k, v = qw.kv_read(s["live"], *cache, dtype=s["k"].dtype)
    return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def own_attn(s):
    import int8_weight_quantized_amd as qw
    return {"out": qw.kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["context"],
                                   s["cu"], s["max_new"], max_context=s["max_context"], window=s["window"])}


def plain_plan(s):
    past, new, B, T = s["past"].long(), s["new"].long(), s["block"], s["total"]
    wide = s["table"].shape[1]
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    have = (past + B - 1) // B
    need = (past + new + B - 1) // B - have
    before = need.cumsum(0) - need
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    pos = past[r] + t - cu[r]
    j = torch.arange(wide, device=DEV)[None, :]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    from_free = s["free"][(before[:, None] + j - have[:, None]).clamp(0, max(0, s["free"].numel() - 1))]
    s["table"].copy_(torch.where(fresh, from_free, s["table"]))
    slots = s["table"][r, pos // B].long() * B + pos % B
    return {"table": s["table"], "cu": cu.int(), "context": (past + new).int(), "positions": pos.int(), "slots": slots.int(),
            "counts": torch.stack((need.sum(), new.sum())).int()}


def plain_rope(s):
    c, si = s["cos"][s["positions"].long()][:, None, :], s["sin"][s["positions"].long()][:, None, :]

    def one(x, weight):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        turned, rest = y[..., :s["rot"]], y[..., s["rot"]:]
        if s["pairs"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack((a * c - b * si, b * c + a * si), -1).flatten(-2)
        else:
            a, b = turned.chunk(2, -1)
            turned = torch.cat((a * c - b * si, b * c + a * si), -1)
        return torch.cat((turned, rest), -1).to(x.dtype)

    return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}


def plain_write(s):
    B, slots, live = s["block"], s["slots"].long(), s["live"].long()
    blk, off = slots // B, slots % B
    lblk, loff = live // B, live % B
    blocks = s["k_scales"].shape[0]
    # the first new place in each block: what lies before it stays
    start = torch.full((blocks,), B, device=DEV).scatter_reduce(0, blk, off, "amin")

    def one(x, codes, scales):
        x = x.float()
        top = torch.zeros_like(scales).scatter_reduce(0, blk[:, None].expand(-1, scales.shape[1]), x.abs().amax(-1), "amax")
        top = top / torch.full_like(top, 127.0)  # by a tensor: a division by a number would multiply by its reciprocal
        top = torch.where(top < TINY, 0.0, top)
        kept = torch.where((start > 0)[:, None], scales, 0.0)
        now = torch.where((start < B)[:, None], torch.maximum(kept, top), scales)
        # codes that stay move to the block's new scale
        ratio = torch.where(now > 0, kept / now, 0.0)[lblk][..., None]
        old = codes[lblk, :, loff]
        moved = torch.where((loff < start[lblk])[:, None, None] & (ratio < 1), torch.round(old.float() * ratio).to(torch.int8), old)
        codes[lblk, :, loff] = moved
        sc = now[blk][..., None]
        codes[blk, :, off] = torch.where(sc > 0, torch.round(x / sc).clamp(-127, 127), 0.0).to(torch.int8)
        scales.copy_(now)
        return (codes[lblk, :, loff].float() * now[lblk][..., None]).to(s["k"].dtype)

    k, v = one(s["k"], s["k_cache"], s["k_scales"]), one(s["v"], s["v_cache"].transpose(2, 3), s["v_scales"])
    return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def plain_attn(s):
    q, table, B = s["q"], s["table"], s["block"]
    T, heads, dim = q.shape
    R, kv, group, n = table.shape[0], s["kv"], heads // s["kv"], s["max_new"]
    table = table[:, :-(-s["max_context"] // B)].long().clamp(min=0)
    k = (s["k_cache"][table].float() * s["k_scales"][table][..., None, None]).transpose(1, 2).reshape(R, kv, -1, dim)
    v = (s["v_cache"][table].float() * s["v_scales"][table][..., None, None]).permute(0, 2, 1, 4, 3).reshape(R, kv, -1, dim)
    cu, context = s["cu"].long(), s["context"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=DEV)[None, :]
    rows = q[(cu[:-1, None] + i).clamp(max=T - 1)].float().view(R, n, kv, group, dim).transpose(1, 2).reshape(R, kv, n * group, dim)
    scores = torch.matmul(rows, k.transpose(2, 3).contiguous()).view(R, kv, n, group, -1) * dim ** -0.5
    j = torch.arange(scores.shape[-1], device=DEV)[None, None, :]
    pos = (context - new)[:, None, None] + i[..., None]
    seen = (j <= pos) & (j < context[:, None, None])
    seen = seen & (j > pos - s["window"]) if s["window"] else seen
    scores = scores.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)  # a row that sees nothing gives zeros
    o = torch.matmul(p.view(R, kv, n * group, -1), v).view(R, kv, n, group, dim).transpose(1, 2).reshape(R, n, heads, dim)
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    return {"out": o[r, t - cu[r]].to(q.dtype)}


PLAIN = {"plan": plain_plan, "rope": plain_rope, "write": plain_write, "attn": plain_attn}
OWN = {"plan": own_plan, "rope": own_rope, "write": own_write, "attn": own_attn}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    def plan(s):
        past, new, table, free, B = s["past"].tolist(), s["new"].tolist(), s["table"].tolist(), s["free"].tolist(), s["block"]
        cu, positions, slots, used = [0], [], [], 0
        for r in range(len(past)):
            cu.append(cu[-1] + new[r])
            for p in range(past[r], past[r] + new[r]):
                if p % B == 0:
                    table[r][p // B] = free[used]
                    used += 1
                positions.append(p)
                slots.append(table[r][p // B] * B + p % B)
        return {"table": ints(table), "cu": ints(cu), "context": ints([p + n for p, n in zip(past, new)]), "positions": ints(positions),
                "slots": ints(slots), "counts": ints([used, cu[-1]])}

    def rope(s):
        rot = s["rot"]
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None, :]
        found = {}
        for n in ("q", "k"):
            x = s[n].double()
            y = s[n + "_weight"].double() * x / ((x * x).sum(-1, keepdim=True) / s["dim"] + 1e-6).sqrt()
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if s["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
            found[n] = y
        return found

    def write(s):
        """Scales are stored in fp32, and codes are the nearest integers (ties to even) to quotients and products that are
        themselves rounded to fp32: both are part of the definition."""
        B, live, slots = s["block"], s["live"].long(), s["slots"].long()
        found = {}
        runs, t = [], 0
        order = slots.tolist()
        while t < len(order):  # a run: the new tokens that fill one block, in order
            end = t + 1
            while end < len(order) and order[end] == order[end - 1] + 1 and order[end] % B:
                end += 1
            runs.append((order[t] // B, order[t] % B, t, end))
            t = end
        for n, cache, scales, x in (("k", s["k_cache"], s["k_scales"], s["k"]), ("v", s["v_cache"].transpose(2, 3), s["v_scales"], s["v"])):
            codes, x = cache.double(), x.double()
            for b, off, lo, hi in runs:
                new = x[lo:hi].transpose(0, 1)  # [kv, tokens, dim]
                scale = (new.abs().amax(dim=(1, 2)) / 127.0).float()
                scale = torch.where(scale < TINY, torch.zeros_like(scale), scale)
                if off:
                    was = scales[b].clone()
                    scale = torch.maximum(scale, was)
                    shrink = torch.where(scale > 0, was.double() / scale.double(), torch.zeros_like(scale).double()).float().double()
                    codes[b, :, :off] = (codes[b, :, :off] * shrink[:, None, None]).float().round().double()
                scales[b] = scale
                safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None, None]
                codes[b, :, off:off + hi - lo] = (new / safe).float().round().clamp(-127, 127).double()
            found[n] = codes[live // B, :, live % B] * scales.double()[live // B][..., None]
            found[n + "_scales"] = scales.double()
        return found

    def attn(s):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        kv, B, dim = s["kv"], s["block"], s["dim"]
        group = s["heads"] // kv
        cu, context, table = s["cu"].tolist(), s["context"].tolist(), s["table"].long()
        for r, c in enumerate(context):
            n = cu[r + 1] - cu[r]
            if c <= 0 or n == 0:
                continue
            ids = table[r, :-(-c // B)]
            low = max(0, c - n - s["window"] + 1) if s["window"] else 0
            pos = torch.arange(c - n, c, device=DEV)[:, None]
            j = torch.arange(low, c, device=DEV)[None, :]
            hidden = (j > pos) | (j <= pos - s["window"]) if s["window"] else j > pos
            for h in range(kv):
                k = (s["k_cache"][ids, h].double() * s["k_scales"][ids, h].double()[:, None, None]).reshape(-1, dim)[low:c]
                v = (s["v_cache"][ids, h].double() * s["v_scales"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, dim)[low:c]
                for g in range(h * group, (h + 1) * group):
                    a = s["q"][cu[r]:cu[r + 1], g].double() @ k.t() / math.sqrt(dim)
                    out[cu[r]:cu[r + 1], g] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ v
        return {"out": out}

    return {"plan": plan, "rope": rope, "write": write, "attn": attn}[case["op"]](prepare(case, seed))
