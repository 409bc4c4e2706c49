"""The attention half of a decoder layer with int8 weights and an int8 cache:
prompts of different lengths, then token after token from a replayed graph.

    python examples/decoder_attention.py [--requests 16] [--prompt 1000] [--tokens 32]

Per step: fused QKV GEMM (int8 weights), plan of the new tokens' places, norm
and rotation of the heads, quantizing write, attention over the cache, output
GEMM.  The last step's output is compared with the same layer in fp32 over
unquantized keys and values.  Weights and activations are random.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import int8_weight_quantized_amd as qw  # noqa: E402


class DecoderAttention:
    """One layer's weights and cache.  The layer owns its requests' block
    table and the list of free blocks; both are advanced on the device."""

    def __init__(self, hidden, heads, kv_heads, head_dim, requests, max_context, block_size=64):
        self.heads, self.kv_heads, self.head_dim, self.block = heads, kv_heads, head_dim, block_size
        width = (heads + 2 * kv_heads) * head_dim
        self.qkv = qw.quantize_weights(torch.randn(width, hidden, device="cuda") * 0.02)
        self.out = qw.quantize_weights(torch.randn(hidden, heads * head_dim, device="cuda") * 0.02)
        self.norms = [(1 + 0.1 * torch.randn(head_dim, device="cuda")).half() for _ in range(2)]
        angle = torch.arange(max_context, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, 1, 2 / head_dim, device="cuda"))
        self.cos, self.sin = angle.cos(), angle.sin()
        columns = -(-max_context // block_size)
        blocks = requests * columns
        self.cache = qw.kv_cache(blocks, kv_heads, head_dim, block_size)
        self.table = torch.full((requests, columns), -1, dtype=torch.int32, device="cuda")
        # in any order; one entry behind the last, so that the list can move on
        self.free = torch.cat([torch.randperm(blocks, device="cuda"), torch.tensor([-1], device="cuda")]).int()
        self.at = torch.arange(blocks + 1, device="cuda")
        self.past = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def project(self, x):
        """q, k and v heads of x [T, hidden], as columns of one matrix."""
        y = qw.w8a16_gemm(x, *self.qkv).view(x.shape[0], -1, self.head_dim)
        return y.split((self.heads, self.kv_heads, self.kv_heads), 1)

    def step(self, x, fresh, max_new):
        """Run the new tokens x [T, hidden] of all requests: fresh[r] (int32)
        tokens of request r, at most max_new."""
        q, k, v = self.project(x)
        plan = qw.kv_plan(self.past, fresh, self.table, self.free, self.block, x.shape[0])
        q, k = qw.qk_norm_rope(q, k, plan.positions, self.cos, self.sin, *self.norms)
        qw.kv_write(k, v, plan.slots, *self.cache)
        o = qw.kv_attention(q, *self.cache, plan.block_table, plan.context, plan.cu_tokens, max_new)
        self.past += fresh
        self.free.copy_(self.free[(self.at + plan.counts[0]).clamp_(max=self.at.shape[0] - 1)])
        return qw.w8a16_gemm(o.view(x.shape[0], -1), *self.out)

    def reference(self, x):
        """The last token's output of one request with tokens x [T, hidden],
        in fp32 with keys and values as projected."""
        q, k, v = (t.float() for t in self.project(x))
        place = torch.arange(x.shape[0], device="cuda")
        half = self.head_dim // 2

        def turn(t, weight):
            t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight.float()
            a, b, c, s = t[..., :half], t[..., half:], self.cos[place, None], self.sin[place, None]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        q, k = turn(q, self.norms[0])[-1], turn(k, self.norms[1])
        group = self.heads // self.kv_heads
        o = []
        for h in range(self.heads):
            weights = torch.softmax(k[:, h // group] @ q[h] * self.head_dim ** -0.5, 0)
            o.append(weights @ v[:, h // group])
        codes, scales = self.out
        return (codes.float() * scales.float()[:, None]) @ torch.cat(o)


def run(hidden=4096, heads=32, kv_heads=2, head_dim=128, requests=16, prompt=1000, tokens=32):
    """Returns (largest error over the largest output, us a prompt step, us a decode step)."""
    torch.manual_seed(0)
    lengths = torch.randint(max(1, prompt // 2), prompt + 1, (requests,))
    layer = DecoderAttention(hidden, heads, kv_heads, head_dim, requests, prompt + tokens + 2)
    prompts = [torch.randn(n, hidden, device="cuda").half() for n in lengths.tolist()]
    steps = [torch.randn(requests, hidden, device="cuda").half() for _ in range(tokens)]
    clock = [torch.cuda.Event(enable_timing=True) for _ in range(4)]

    packed, fresh = torch.cat(prompts), lengths.to(torch.int32).cuda()
    DecoderAttention(hidden, heads, kv_heads, head_dim, requests, prompt + tokens + 2).step(packed, fresh, int(lengths.max()))
    clock[0].record()  # (behind one like it, which loads the kernels)
    layer.step(packed, fresh, int(lengths.max()))
    clock[1].record()

    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    x = steps[0].clone()
    layer.step(x, one, 1)  # the first token eagerly, the others from a graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x, one, 1)
    clock[2].record()
    for s in steps[1:]:
        x.copy_(s)
        graph.replay()
    clock[3].record()
    torch.cuda.synchronize()

    worst = top = 0.0
    for r in {0, requests // 2, requests - 1}:
        want = layer.reference(torch.cat([prompts[r]] + [s[r:r + 1] for s in steps]))
        worst = max(worst, (y[r].float() - want).abs().max().item())
        top = max(top, want.abs().max().item())
    assert layer.past.tolist() == (lengths + tokens).tolist()
    return worst / top, clock[0].elapsed_time(clock[1]) * 1e3, clock[2].elapsed_time(clock[3]) * 1e3 / max(1, tokens - 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--prompt", type=int, default=1000, help="longest prompt; the shortest is half of it")
    p.add_argument("--tokens", type=int, default=32)
    a = p.parse_args()
    if min(a.requests, a.prompt, a.tokens - 1) < 1:
        p.error("needs a request, a prompt token and two tokens")
    error, prompt_us, token_us = run(requests=a.requests, prompt=a.prompt, tokens=a.tokens)
    print("%d requests, prompts of %d to %d tokens: %.0f us for the prompts' step, %.1f us a decode step, error %.2g of the largest output"
          % (a.requests, max(1, a.prompt // 2), a.prompt, prompt_us, token_us, error))


if __name__ == "__main__":
    main()
