"""The feed-forward half of a decoder layer with int8 weights: a prompt, then
decode steps from a replayed graph, once with one product for all tokens and
once with experts.

    python examples/decoder_feed_forward.py [--tokens 16] [--prompt 1000] [--steps 32]

Dense: residual addition and norm, gated gate-and-up product, down product onto
the residual stream; --codes passes the activations as int8 (W8A8).  Experts: the
same norm, the router's logits, the route, the experts' gated and down products
in the route's order, and their weighted sum onto the residual stream.  The last
step's output is compared with the same layer in fp32.  Weights and activations
are random.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import int8_weight_quantized_amd as qw  # noqa: E402


def weights(*shape):
    """Random int8 codes and scales: [..., channels, inputs]."""
    flat = qw.quantize_weights(torch.randn(shape, device="cuda").view(-1, shape[-1]) * shape[-1] ** -0.5)
    return flat[0].view(shape), flat[1].view(shape[:-1])


def real(q, s):
    return q.float() * s.float()[..., None]


def norm32(x, residual, weight):
    h = (x.float() + residual.float()).half().float()
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * weight.float(), h


class Dense:
    def __init__(self, hidden, inner, codes):
        self.norm = (1 + 0.1 * torch.randn(hidden, device="cuda")).half()
        self.up, self.down, self.codes = weights(2 * inner, hidden), weights(hidden, inner), codes

    def __call__(self, x, residual):
        if self.codes:
            q, s, h = qw.add_rms_norm(x, self.norm, residual, quantize=True)
            g = qw.w8a8_linear(q, s, *self.up, activation="silu", gated=True)
            return qw.w8a8_linear(*qw.quantize_activations(g), *self.down, residual=h)
        y, h = qw.add_rms_norm(x, self.norm, residual)
        return qw.w8a16_linear(qw.w8a16_linear(y, *self.up, activation="silu", gated=True), *self.down, residual=h)

    def reference(self, x, residual):
        y, h = norm32(x, residual, self.norm)
        gate, up = (y @ real(*self.up).t()).chunk(2, 1)
        return h + (torch.nn.functional.silu(gate) * up) @ real(*self.down).t()


class Experts:
    def __init__(self, hidden, inner, experts, top_k):
        self.norm = (1 + 0.1 * torch.randn(hidden, device="cuda")).half()
        self.router = (torch.randn(hidden, experts, device="cuda") * hidden ** -0.5).half()
        self.up, self.down, self.top_k = weights(experts, 2 * inner, hidden), weights(experts, hidden, inner), top_k

    def __call__(self, x, residual):
        y, h = qw.add_rms_norm(x, self.norm, residual)
        self.route = qw.route_experts(y @ self.router, self.top_k)
        g = qw.w8a16_experts(y, *self.up, self.route, activation="silu", gated=True)
        d = qw.w8a16_experts(g, *self.down, self.route, gather=False, dtype=torch.float32)
        return qw.experts_combine(d, self.route, residual=h)

    def reference(self, x, residual):
        """With the route as taken: a token whose choices are close may take
        another one in fp32."""
        y, out = norm32(x, residual, self.norm)
        for t, (ids, shares) in enumerate(zip(self.route.ids.tolist(), self.route.weights)):
            for e, share in zip(ids, shares):
                gate, up = (real(self.up[0][e], self.up[1][e]) @ y[t]).chunk(2)
                out[t] += share * (real(self.down[0][e], self.down[1][e]) @ (torch.nn.functional.silu(gate) * up))
        return out


def run(layer, hidden, tokens=16, prompt=1000, steps=32):
    """Returns (largest error over the largest output, us a prompt, us a decode step)."""
    clock = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    x, h = (torch.randn(prompt, hidden, device="cuda").half() for _ in range(2))
    layer(x, h)
    clock[0].record()  # (behind one like it, which loads the kernels)
    layer(x, h)
    clock[1].record()

    x, h = (torch.randn(tokens, hidden, device="cuda").half() for _ in range(2))
    inputs = [torch.randn_like(x) for _ in range(steps)]
    layer(x, h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, h)
    clock[2].record()
    for step in inputs:
        x.copy_(step)
        graph.replay()
    clock[3].record()
    torch.cuda.synchronize()
    want = layer.reference(x, h)
    error = ((y.float() - want).abs().max() / want.abs().max()).item()
    return error, clock[0].elapsed_time(clock[1]) * 1e3, clock[2].elapsed_time(clock[3]) * 1e3 / max(1, steps)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=16, help="of a decode step")
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--codes", action="store_true", help="int8 activations in the dense layer")
    a = p.parse_args()
    if min(a.tokens, a.prompt, a.steps) < 1:
        p.error("needs a token, a prompt token and a step")
    torch.manual_seed(0)
    for name, hidden, layer in (("one product, 4096 by 13696", 4096, Dense(4096, 13696, a.codes)),
                                ("8 of 64 experts, 2048 by 1024", 2048, Experts(2048, 1024, 64, 8))):
        error, prompt_us, step_us = run(layer, hidden, a.tokens, a.prompt, a.steps)
        print("%s: %.0f us for a prompt of %d, %.1f us a decode step of %d, error %.2g of the largest output"
              % (name, prompt_us, a.prompt, step_us, a.tokens, error))


if __name__ == "__main__":
    main()
