"""One feed-forward layer with 8-bit activations throughout, as a server runs it on a residual
stream:

    h = h + y (y: the layer before), x = norm(h), out = down(silu(gate x) * (up x))

in two forms: e4m3 weights with a scale for each block of 128 x 128, and K-quant weights (gate and up
q4_K, down q6_K) with int8 activations. Norm, gated activation and products hand each other codes
and scales; nothing is quantised in a pass of its own.

    python examples/feed_forward.py              # one decoded token, a decode batch, a prompt
    python examples/feed_forward.py --check      # small sizes against 64 bits

Weights are random.
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import q6_int8_mmq_gb300 as q6  # noqa: E402
from examples.moe_layer import dequantise, random_blocks  # noqa: E402

EPS = 1e-6


class BlockLayer:
    """e4m3 weights; y and the result bf16, the stream bf16."""

    def __init__(self, hidden, inner, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen)).bfloat16().cuda()
        self.dense = {
            "up": (torch.randn(2 * inner, hidden, generator=gen) / math.sqrt(hidden)).bfloat16().cuda(),
            "down": (torch.randn(hidden, inner, generator=gen) / math.sqrt(inner)).bfloat16().cuda()}
        self.up, self.down = (q6.f8_quantize_weights(self.dense[k]) for k in ("up", "down"))

    def __call__(self, y, h):
        """Adds y to the stream h in place and returns the layer's output."""
        x, h = q6.rms_norm_f8(y, self.norm, EPS, residual=h)
        gate_up, _ = q6.f8_mmq(self.up, x)
        return q6.f8_mmq(self.down, q6.silu_mul_f8(gate_up))[0]

    def weights(self):
        return self.dense["up"].double(), self.dense["down"].double()


class KQuantLayer:
    """q4_K gate and up, q6_K down; y, the stream and the result f32."""

    def __init__(self, hidden, inner, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen)).cuda()
        self.raw = {"up": random_blocks("q4_K", 1, 2 * inner, hidden, gen)[0].cuda(),
                    "down": random_blocks("q6_K", 1, hidden, inner, gen)[0].cuda()}
        self.up = q6.q4k_pack_weights(self.raw["up"].view(-1), 2 * inner, hidden, wq=True)
        self.down = q6.pack_weights(self.raw["down"].view(-1), hidden, inner, wh=True)

    def __call__(self, y, h):
        x, h = q6.rms_norm_q8(y, self.norm, EPS, residual=h, want_us=True)
        gate_up, _, _ = q6.q4k_mmq(self.up, x)
        return q6.mmq(self.down, q6.silu_mul_q8(gate_up))[0]

    def weights(self):
        return dequantise(self.raw["up"], "q4_K"), dequantise(self.raw["down"], "q6_K")


def exact(layer, y, h):
    """The layer in 64 bits from the unquantised activations: (output, stream)."""
    up, down = layer.weights()
    h = h.double() + y.double()
    x = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * layer.norm.double()
    gate, u = (x @ up.t()).chunk(2, dim=1)
    return (gate * torch.sigmoid(gate) * u) @ down.t(), h


def inputs(layer, tokens, hidden, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = layer.norm.dtype
    return [torch.randn(tokens, hidden, device="cuda", generator=gen).to(dtype) for _ in range(2)]


def check(layer, tokens, hidden):
    """The layer's distance from 64 bits, relative to the result's size."""
    y, h = inputs(layer, tokens, hidden)
    want, stream = exact(layer, y, h)
    got = layer(y, h).double()
    q6.sync_status()
    assert (h.double() - stream).norm() <= 2.0 ** -8 * stream.norm()
    return ((got - want).norm() / want.norm()).item()


def time_layer(layer, tokens, hidden, steps=50):
    y, h = inputs(layer, tokens, hidden)
    for _ in range(5):
        layer(y, h)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        layer(y, h)
    end.record()
    end.synchronize()
    q6.sync_status()
    return begin.elapsed_time(end) * 1e3 / steps


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--check", action="store_true", help="compare small sizes with 64 bits")
    a = p.parse_args(argv)
    for cls, name in ((BlockLayer, "e4m3 blocks"), (KQuantLayer, "q4_K and q6_K")):
        hidden, inner = (512, 768) if a.check else (4096, 11008)
        layer = cls(hidden, inner)
        for tokens in (1, 5, 200) if a.check else (1, 32, 2048):
            if a.check:
                print(f"{name}, {tokens} tokens: {check(layer, tokens, hidden):.2e} from 64 bits")
            else:
                print(f"{name}, {tokens:5d} tokens, {inner} x {hidden}: "
                      f"{time_layer(layer, tokens, hidden):8.1f} us")


if __name__ == "__main__":
    main()
