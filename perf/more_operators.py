"""Cases and plain forms of the 8-bit steps around the projections: the norm and the gated
activation that end in quantised activations, the quantisers of 8-bit floating point, and the
matrix product of such blocks.

Four operators, named by a case's "op":

norm      h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, given as 8-bit codes and
          scales, and h, the residual stream that goes on.
silu      y = silu(gate) * up of rows that hold gate then up, given as codes and scales.
quantise  rows of activations (a scale for each 128 of a row) or a weight matrix (a scale for
          each block of 128 x 128) as e4m3 codes and scales.
product   Y[n][m] = sum over blocks b of sx[b][n] * sw[m / 128][b] * (sum over k in b of
          xq[n][k] * wq[m][k]), xq and wq e4m3 codes.

Codes ("to"):
  q8  int8, a scale for each 32 of a row: scale = largest / 127, code = value / scale rounded,
      halves away from zero; as int8 and as the binary16 operand plane of the tensor cores.
  f8  e4m3, a scale for each 128: scale = largest / 448, code = value * (448 / largest) rounded.
The norm's codes are those of h * weight: 1 / sqrt(mean(h^2) + eps) is a factor of the whole row
and goes into its scales.

own selects the framework's kernels; otherwise everything runs as elementary torch operations in
32 bits, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decoded token between two projections of K-quant weights: latency alone counts
        dict(name="norm one token q8", op="norm", to="q8", N=1, K=4096, type="f32", rtype="f32"),
        # a prompt's f32 residual stream on its way into the prefill product
        dict(name="norm prompt q8", op="norm", to="q8", N=3314, K=4096, type="f32", rtype="f32"),
        # a decode batch of odd size, bf16 throughout
        dict(name="norm decode batch f8", op="norm", to="f8", N=47, K=3584, type="bf16",
             rtype="bf16"),
        # a long prompt, the first norm of a model apart: bf16 sublayer output on a bf16 stream
        dict(name="norm long prompt f8", op="norm", to="f8", N=8192, K=4096, type="bf16",
             rtype="bf16"),
        # one decoded token between the up and the down projection
        dict(name="silu one token f8", op="silu", to="f8", N=1, K=11008, type="bf16"),
        # a prompt's f32 gate and up outputs on their way into the K-quant down projection
        dict(name="silu prompt q8", op="silu", to="q8", N=3314, K=11008, type="f32"),
        # a prompt of odd size into an 8-bit product
        dict(name="quantise prompt", op="quantise", what="act", N=3325, K=3584, type="f16"),
        # a weight matrix of a checkpoint, once at load time
        dict(name="quantise weight", op="quantise", what="weight", N=11008, K=4096, type="bf16"),
        # one decoded token's widest projection
        dict(name="product one token", op="product", N=1, M=11008, K=4096, type="bf16"),
        # a decode batch of odd size, the down projection
        dict(name="product decode batch", op="product", N=33, M=4096, K=11008, type="f16"),
        # a short prompt with ragged ends: rows, columns and K are no multiples of a block
        dict(name="product ragged prompt", op="product", N=1023, M=2056, K=3600, type="f32"),
        # a long prompt's gate and up projections in one
        dict(name="product long prompt", op="product", N=8192, M=22016, K=4096, type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "silu", "quantise", "product", "product"])
    types = ["f32", "bf16", "f16"]
    if op in ("norm", "silu"):
        to = rng.choice(["q8", "f8"])
        K = 256 * _log_int(rng, 1, 43) if to == "q8" else 16 * _log_int(rng, 4, 688)
        case = dict(op=op, to=to, N=min(_log_int(rng, 1, 8192), 8192 * 4096 // K), K=K,
                    type=rng.choice(types))
        if op == "norm":
            case["rtype"] = rng.choice(["none", "f32", case["type"]])
        return case
    if op == "quantise":
        K = 16 * _log_int(rng, 4, 688)
        return dict(op=op, what=rng.choice(["act", "weight"]),
                    N=min(_log_int(rng, 1, 11008), 11008 * 4096 // K), K=K, type=rng.choice(types))
    M, K = _log_int(rng, 64, 22016), 16 * _log_int(rng, 4, 688)
    return dict(op=op, N=min(_log_int(rng, 1, 8192), 8192 * 22016 * 4096 // (M * K)), M=M, K=K,
                type=rng.choice(types))


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    N, K = c["N"], c["K"]
    blocks = -(-K // 128)
    if c["op"] == "product":
        M = c["M"]
        return {"bytes": (N + M) * K + 4 * blocks * (N + -(-M // 128)) + N * M * size[c["type"]],
                "flops": 2 * N * M * K}
    if c["op"] == "quantise":
        rows = N if c["what"] == "act" else -(-N // 128)
        return {"bytes": N * K * (size[c["type"]] + 1) + 4 * rows * blocks, "flops": 3 * N * K}
    # codes and scales: q8 as int8 (the norm's) and binary16, f8 as e4m3
    if c["to"] == "q8":
        out = N * K * (3 if c["op"] == "norm" else 2) + N * K // 8
    else:
        out = N * K + 4 * N * blocks
    if c["op"] == "silu":
        return {"bytes": 2 * N * K * size[c["type"]] + out, "flops": 8 * N * K}
    return {"bytes": N * K * (size[c["type"]] + 2 * size[c["rtype"]]) + 2 * K + out,
            "flops": 7 * N * K}


# ----------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, N, K):
    """N(0, 1) with one channel in a hundred 20 times larger, as a model's activations have."""
    wide = torch.rand(K, generator=g, device="cuda") < 0.01
    return _randn(g, N, K) * torch.where(wide, 20.0, 1.0)


def _weights(g, M, K):
    """About N(0, 1 / K), blocks of 128 x 128 of sizes of their own."""
    vary = torch.exp(0.3 * _randn(g, -(-M // 128), -(-K // 128)))
    vary = vary.repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    return _randn(g, M, K) * vary / math.sqrt(K)


def _inputs(case, seed):
    """The tensors both forms start from, made from the seed alone."""
    c, g = case, _gen(seed)
    N, K = c["N"], c["K"]
    if c["op"] == "norm":
        x = _activations(g, N, K).to(DTYPES[c["type"]])
        weight = (1 + 0.2 * _randn(g, K)).bfloat16()
        r = (3 * _activations(g, N, K)).to(DTYPES[c["rtype"]]) if c["rtype"] != "none" else None
        return dict(x=x, residual=r, weight=weight)
    if c["op"] == "silu":
        return dict(x=(1.5 * _activations(g, N, 2 * K)).to(DTYPES[c["type"]]))
    if c["op"] == "quantise":
        make = _activations if c["what"] == "act" else _weights
        return dict(x=make(g, N, K).to(DTYPES[c["type"]]))
    xq, sx = _f8_rows(_activations(g, N, K))
    wq, sw = _f8_blocks(_weights(g, c["M"], K))
    # scales of a block next to each other, rows of them 16 bytes apart or a multiple of that
    rows = torch.zeros(sx.shape[0], -(-N // 4) * 4, device="cuda")
    rows[:, :N] = sx
    return dict(xq=xq, sx=rows, wq=wq, sw=sw)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = c = case
    if own:
        import q6_int8_mmq_gb300 as q6
        dev = torch.device("cuda")
        if c["op"] == "product":
            s["w"] = q6.F8Weights(c["M"], c["K"], s["wq"], s["sw"])
            s["act"] = q6.F8Activations(c["N"], c["K"], s["xq"], s["sx"])
            s["out"] = torch.empty((c["N"], c["M"]), dtype=DTYPES[c["type"]], device=dev)
        elif c["op"] == "quantise" and c["what"] == "weight":
            s["out"] = q6.alloc_f8_weights(c["N"], c["K"], dev)
        elif c["op"] == "quantise" or c["to"] == "f8":
            s["out"] = q6.alloc_f8_activations(c["N"], c["K"], dev)
        else:
            s["out"] = q6.alloc_activations(c["N"], c["K"], dev, want_xq=c["op"] == "norm")
        if c["op"] == "norm" and s["residual"] is not None:
            s["h"] = torch.empty_like(s["residual"])
    return s


# ------------------------------------------------------------ plain forms ---

def _by(a, b):
    """a / b element by element; a number may be either (a division by a number itself would be
    a product with its rounded reciprocal)."""
    full = a if isinstance(a, torch.Tensor) else b
    a, b = (v if isinstance(v, torch.Tensor) else torch.full_like(full, v) for v in (a, b))
    return a / b


def _q8_rows(t):
    """f32 [N, K] -> codes as f32 [N, K], scales [K / 32, N]."""
    b = t.unflatten(1, (-1, 32))
    d = _by(b.abs().amax(2), 127.0)
    q = torch.where(d.unsqueeze(2) > 0, b / d.unsqueeze(2), 0.0)
    low = q.abs().floor()
    q = (low + (q.abs() - low >= 0.5)).clamp(max=127).copysign(q)
    return q.flatten(1), d.t()


def _f8(b, top):
    """Blocks b with their largest magnitudes -> e4m3 codes and scales."""
    live = top >= 2.0 ** -100
    up = torch.where(live, _by(448.0, top), 0.0)
    return (b * up).to(torch.float8_e4m3fn), torch.where(live, _by(top, 448.0), 0.0)


def _f8_rows(t):
    """f32 [N, K] -> e4m3 [N, K], scales [K / 128 rounded up, N]."""
    N, K = t.shape
    b = torch.nn.functional.pad(t, (0, -K % 128)).unflatten(1, (-1, 128))
    q, s = _f8(b, b.abs().amax(2, keepdim=True))
    return q.flatten(1)[:, :K].contiguous(), s.squeeze(2).t()


def _f8_blocks(t):
    """f32 [M, K] -> e4m3 [M, K], scales [M / 128, K / 128], both rounded up."""
    M, K = t.shape
    b = torch.nn.functional.pad(t, (0, -K % 128, 0, -M % 128))
    b = b.unflatten(1, (-1, 128)).unflatten(0, (-1, 128))          # [M', 128, K', 128]
    q, s = _f8(b, b.abs().amax((1, 3), keepdim=True))
    return q.flatten(2).flatten(0, 1)[:M, :K].contiguous(), s[:, 0, :, 0].contiguous()


def _norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    t = h * s["weight"].float()
    r = torch.rsqrt(h.square().mean(1) + EPS)                       # of each row
    if c["to"] == "q8":
        q, d = _q8_rows(t)
        out = {"xq": q.to(torch.int8), "xh": q.half(), "scale": d * r}
    else:
        q, d = _f8_rows(t)
        out = {"codes": q, "scale": d * r}
    if s["residual"] is not None:
        out["h"] = h.to(s["residual"].dtype)
    return out


def _silu(s):
    gate, up = s["x"].float().chunk(2, dim=1)
    y = gate / (1 + torch.exp(-gate)) * up
    if s["case"]["to"] == "q8":
        q, d = _q8_rows(y)
        return {"xh": q.half(), "scale": d}
    q, d = _f8_rows(y)
    return {"codes": q, "scale": d}


def _quantise(s):
    q, d = (_f8_rows if s["case"]["what"] == "act" else _f8_blocks)(s["x"].float())
    return {"codes": q, "scale": d}


def _product(s):
    c = s["case"]
    N, M, K = c["N"], c["M"], c["K"]
    x = s["xq"].float() * s["sx"][:, :N].t().repeat_interleave(128, 1)[:, :K]
    w = s["wq"].float() * s["sw"].repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    return (x @ w.t()).to(DTYPES[c["type"]])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "silu": _silu, "quantise": _quantise, "product": _product}[c["op"]](s)
    import q6_int8_mmq_gb300 as q6
    if c["op"] == "product":
        return q6.f8_mmq(s["w"], s["act"], out=s["out"])[0]
    if c["op"] == "quantise":
        if c["what"] == "weight":
            w = q6.f8_quantize_weights(s["x"], out=s["out"])
            return {"codes": w.wq, "scale": w.sw}
        act = q6.f8_quantize_act(s["x"], out=s["out"])
    elif c["op"] == "silu":
        act = (q6.silu_mul_q8 if c["to"] == "q8" else q6.silu_mul_f8)(s["x"], out=s["out"])
    else:
        norm = q6.rms_norm_q8 if c["to"] == "q8" else q6.rms_norm_f8
        act, h = norm(s["x"], s["weight"], EPS, residual=s["residual"], h=s.get("h"), out=s["out"])
    if c.get("to") == "q8":
        out = {"xh": act.xh, "scale": act.da[:, :c["N"]]}
        if c["op"] == "norm":
            out["xq"] = act.xq
    else:
        out = {"codes": act.xq, "scale": act.sx[:, :c["N"]]}
    if c["op"] == "norm" and s["residual"] is not None:
        out["h"] = h
    return out


# ---------------------------------------------------------------- 64 bits ---

def _exact_f8(v, group):
    """The e4m3 values nearest to 448 v / largest, ties to even, and largest / 448; `group`:
    the number of each element's block. Returns values shaped as v, and a scale for each block."""
    n = int(group.max()) + 1
    top = torch.zeros(n, dtype=torch.float64, device=v.device)
    top = top.scatter_reduce(0, group.reshape(-1), v.abs().reshape(-1), "amax")
    up = torch.where(top > 0, 448 / top, 0.0)
    u = v * up[group]
    step = torch.ldexp(torch.ones_like(u), (torch.frexp(u)[1] - 4).clamp(min=-9))
    return torch.round(u / step) * step, top / 448


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    N, K = c["N"], c["K"]
    if c["op"] == "product":
        at = torch.arange(K, device="cuda") // 128
        x = s["xq"].double() * s["sx"].double()[at][:, :N].t()
        mt = torch.arange(c["M"], device="cuda") // 128
        w = s["wq"].double() * s["sw"].double()[mt][:, at]
        return x @ w.t()
    v, root, h = s["x"].double(), None, None
    if c["op"] == "norm":
        h = v if s["residual"] is None else v + s["residual"].double()
        root = ((h * h).sum(1) / K + EPS) ** 0.5
        v = h * s["weight"].double()
    elif c["op"] == "silu":
        v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
    row = torch.arange(N, device="cuda").unsqueeze(1)
    col = torch.arange(K, device="cuda").unsqueeze(0)
    if c.get("to") == "q8":
        b = v.view(N, K // 32, 32)
        scale = b.abs().max(2)[0] / 127
        q = torch.where(scale.unsqueeze(2) > 0, b / scale.unsqueeze(2), 0.0)
        q = (torch.sign(q) * torch.floor(q.abs() + 0.5)).view(N, K)
        scale = scale if root is None else scale / root.unsqueeze(1)
        out = {"xh": q, "scale": scale.t()}
        if c["op"] == "norm":
            out["xq"] = None                       # the same codes as xh, as whole numbers
    else:
        weight = c["op"] == "quantise" and c["what"] == "weight"
        wide = -(-K // 128)
        q, scale = _exact_f8(v, (row // 128 if weight else row) * wide + col // 128)
        scale = scale.view(-1, wide)
        scale = scale if root is None else scale / root.unsqueeze(1)
        out = {"codes": q, "scale": scale if weight else scale.t()}
    if h is not None and s["residual"] is not None:
        out["h"] = h
    return out
