"""One mixture-of-experts layer from K-quant weights, as a server runs it for a batch of requests:

    out = shared projection (q6_K x int8) + each request's low-rank adapter
          + the chosen experts' silu(gate) * up and down products (q4_K and q6_K), weighted

    python examples/moe_layer.py                 # one decoded token, a decode batch, a prompt
    python examples/moe_layer.py --check         # small sizes against 64 bits

Weights are random; the router's own product is a plain matrix product.
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


def random_blocks(fmt, experts, rows, cols, gen):
    """K-quant bytes whose weights are about N(0, 1 / cols) in size."""
    size = {"q4_K": 144, "q6_K": 210}[fmt]
    raw = torch.randint(0, 256, (experts, rows, cols // 256, size), generator=gen, dtype=torch.uint8)
    d = torch.full(raw.shape[:3] + (1,), (1 / 170 if fmt == "q4_K" else 1 / 1370) / math.sqrt(cols))
    if fmt == "q4_K":
        raw[..., 0:2] = d.half().view(torch.uint8)
        raw[..., 2:4] = (7.5 * d).half().view(torch.uint8)
    else:
        raw[..., 208:210] = d.half().view(torch.uint8)
    return raw


class MoeLayer:
    """hidden wide, `experts` experts of `inner` features (topk a token), a shared hidden x hidden
    projection with `adapters` low-rank adapters."""

    def __init__(self, hidden, inner, experts, topk, adapters, rank, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.topk, self.experts, self.n_adapters = topk, experts, adapters
        self.raw = {"shared": random_blocks("q6_K", 1, hidden, hidden, gen)[0].cuda(),
                    "up": random_blocks("q4_K", experts, 2 * inner, hidden, gen).cuda(),
                    "down": random_blocks("q6_K", experts, hidden, inner, gen).cuda()}
        self.router = (torch.randn(experts, hidden, generator=gen) / math.sqrt(hidden)).cuda()
        self.shared = q6.pack_weights(self.raw["shared"].view(-1), hidden, hidden, wh=True)
        self.up = q6.pack_experts(self.raw["up"], "q4_K", experts, 2 * inner, hidden, swiglu=True)
        self.down = q6.pack_experts(self.raw["down"], "q6_K", experts, hidden, inner)
        a = torch.randn(adapters, rank, hidden, generator=gen) / math.sqrt(hidden)
        b = torch.randn(adapters, hidden, rank, generator=gen) / math.sqrt(rank)
        self.adapters = q6.LoraAdapters(a.bfloat16().cuda(), b.bfloat16().cuda(),
                                        torch.full((adapters,), 0.5).cuda())

    def __call__(self, x, requests):
        """x [N, hidden] f32; requests: the grouping of the tokens by adapter, made once a step
        for all layers. Returns bf16 [N, hidden]."""
        y, _, _ = q6.mmq(self.shared, q6.quantize_act(x))
        q6.lora_add(self.adapters, x, requests, y)
        route = q6.moe_route(x @ self.router.t(), self.topk)
        h, _ = q6.experts_mmq(self.up, x.bfloat16(), route.groups)
        h, _ = q6.experts_mmq(self.down, h, route.groups, gather=False)
        return q6.moe_combine(h, route.groups.pos, route.weights, shared=y)


def time_layer(layer, hidden, tokens, steps=50):
    x = torch.randn(tokens, hidden, device="cuda")
    ids = torch.randint(-1, layer.n_adapters, (tokens,), device="cuda").sort()[0].int()
    requests = q6.group_rows(ids, layer.n_adapters)
    for _ in range(5):
        layer(x, requests)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        layer(x, requests)
    end.record()
    end.synchronize()
    q6.sync_status()
    return begin.elapsed_time(end) * 1e3 / steps


def dequantise(raw, fmt):
    """f64 weights of raw blocks [..., blocks, bytes]."""
    k = torch.arange(256, device=raw.device)
    half = lambda b: b.contiguous().view(torch.float16).double()  # noqa: E731
    if fmt == "q4_K":
        j = k // 32
        q = (raw[..., 16 + 32 * (j // 2) + k % 32].int() >> (4 * (j % 2)).int()) & 15
        a, m, l = (raw[..., o + 4 + j % 4].int() for o in (0, 4, 8))
        sc = torch.where(j < 4, a & 63, (l & 15) | ((a >> 6) << 4))
        mn = torch.where(j < 4, m & 63, (l >> 4) | ((m >> 6) << 4))
        return (half(raw[..., 0:2]) * (sc * q) - half(raw[..., 2:4]) * mn).flatten(-2)
    h, r = k // 128, k % 128
    q = (raw[..., 64 * h + r % 64].int() >> (4 * (r // 64)).int()) & 15
    q |= ((raw[..., 128 + 32 * h + r % 32].int() >> (2 * (r // 32)).int()) & 3) << 4
    sc = raw[..., 192 + k // 16].contiguous().view(torch.int8).double()
    return (half(raw[..., 208:210]) * sc * (q - 32)).flatten(-2)


def exact(layer, x, ids):
    """The layer in 64 bits (without the shared projection's int8 rounding of x)."""
    x = x.double()
    out = x @ dequantise(layer.raw["shared"], "q6_K").t()
    a, b = layer.adapters.A.double(), layer.adapters.B.double()
    for n, i in enumerate(ids.tolist()):
        if i >= 0:
            out[n] += 0.5 * (b[i] @ (a[i] @ x[n]))
    best, chosen = (x.float() @ layer.router.t()).double().topk(layer.topk, dim=1)
    weights = torch.softmax(best, 1)
    for e in range(layer.experts):
        n, slot = (chosen == e).nonzero(as_tuple=True)
        gate, up = (x[n] @ dequantise(layer.raw["up"][e], "q4_K").t()).chunk(2, dim=1)
        y = (gate * torch.sigmoid(gate) * up) @ dequantise(layer.raw["down"][e], "q6_K").t()
        out.index_add_(0, n, weights[n, slot, None] * y)
    return out


def check(tokens, hidden=512, inner=256, experts=8):
    """The layer's distance from 64 bits, relative to the result's size."""
    layer = MoeLayer(hidden, inner, experts, 2, 3, 16)
    x = torch.randn(tokens, hidden, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    ids = (torch.arange(tokens, device="cuda") % 4 - 1).int()
    got = layer(x, q6.group_rows(ids, 3)).double()
    q6.sync_status()
    want = exact(layer, x, ids)
    return ((got - want).norm() / want.norm()).item()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--check", action="store_true", help="compare small sizes with 64 bits")
    a = p.parse_args(argv)
    if a.check:
        for tokens in (1, 5, 200):
            print(f"{tokens} tokens: {check(tokens):.2e} from 64 bits")
        return
    hidden, inner, experts, topk = 2048, 768, 64, 8
    layer = MoeLayer(hidden, inner, experts, topk, adapters=8, rank=16)
    for tokens in (1, 32, 2048):
        print(f"{tokens:5d} tokens, {topk} of {experts} experts of {inner} x {hidden}: "
              f"{time_layer(layer, hidden, tokens):8.1f} us")


if __name__ == "__main__":
    main()
