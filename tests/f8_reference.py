"""64-bit references of the 8-bit steps around the projections, from their definitions, with the
error bounds the tests hold the kernels to. All tensors are torch's, on any device.

Unit roundoffs: f32 2^-24, bf16 2^-8, f16 2^-11, e4m3 2^-4 (half a step relative to the value; half
of the smallest subnormal step, 2^-10, below 2^-6)."""
import torch

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half of the smallest subnormal step (bf16's and f32's are below what the tests use)
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def block_max(t, side_rows, side_cols):
    """max|t| of the blocks of a matrix, and each element's: [rows', cols'], [rows, cols]."""
    M, K = t.shape
    top = torch.nn.functional.pad(t.abs(), (0, -K % side_cols, 0, -M % side_rows))
    top = top.unflatten(1, (-1, side_cols)).unflatten(0, (-1, side_rows)).amax((1, 3))
    each = top.repeat_interleave(side_rows, 0)[:M].repeat_interleave(side_cols, 1)[:, :K]
    return top, each


def check_codes(codes, scale, t, rel, root, root_rel, f8, rows=1):
    """codes [N, K] and scale [N', K'] (as f64) against t [N, K] f64 that the kernel knows within
    rel (a tensor or number, relative); root: the rows' factor [N, 1] (or 1.0) within root_rel.

    A code is its block's t / d (e4m3: t * (448 / max)) within half a step; t and max are within
    rel of the exact ones, and d and the quotient add two roundings of f32 each."""
    top, each = block_max(t, rows, 128 if f8 else 32)
    rel = rel + torch.zeros_like(t)
    d = each / (448.0 if f8 else 127.0)
    live = each >= 2.0 ** -100 if f8 else each > 0
    u = torch.where(live, t / d, 0.0)
    _, top_rel = block_max(torch.where(t.abs() >= 0.99 * each, rel, 0.0), rows, 128 if f8 else 32)
    slack = u.abs() * (rel + top_rel + 4 * U)
    half = (u.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) if f8 else 0.5
    off = (codes - u).abs()
    assert (off <= half + slack).all(), float((off - half - slack).max())
    # 2^e boundaries: a step is twice as long above, so a code is within half of the larger one
    want = top / (448.0 if f8 else 127.0) * root
    dead = top < 2.0 ** -100 if f8 else top == 0
    want = torch.where(dead, 0.0, want)
    bound = want.abs() * (float(rel.max()) + 4 * U + root_rel)
    assert ((scale - want).abs() <= bound).all(), float(((scale - want).abs() - bound).max())


def norm(x, residual, weight, eps):
    """(h, t, root, rel, root_rel): t = h * weight within rel, root = 1 / sqrt(mean(h^2) + eps)
    within root_rel. In f32 h and t are rounded once each. A row's squares (each with h's rounding
    twice and one of its own) are summed in chains of at most K / 256 + 8 + 5 + 32 additions, the
    root halves that and adds its own rounding, the division's and the sum's with eps."""
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    root = ((h * h).mean(1, keepdim=True) + eps) ** -0.5
    K = x.shape[1]
    return h, h * weight.double(), root, 2 * U, ((K / 256 + 45 + 3) / 2 + 4) * U


def silu_mul(x):
    """(t, rel): silu(gate) * up within rel: the exponential is off by 2 + 1.2 |g| units of 2^-23
    (its share of 1 + exp(-g) is at most all of it), the addition, division and product by
    1/2, 2 and 1/2."""
    g, u = x.double().chunk(2, dim=1)
    rel = (5 + 1.2 * g.abs()) * 2.0 ** -23
    return g * torch.sigmoid(g) * u, rel


def product(xq, sx, wq, sw, dtype):
    """(Y, bound): xq [N, K], wq [M, K] e4m3; sx [K', >= N], sw [M', K'].

    Within a block each of the 128 products and 4 intermediate sums may lose 2^-24 of the largest
    by truncation; the scales' product and one fused multiply-add a block add 2^-24 each, then
    the sum is rounded to dtype."""
    N, K = xq.shape
    M = wq.shape[0]
    x = xq.double() * sx[:, :N].double().t().repeat_interleave(128, 1)[:, :K]
    w = wq.double() * sw.double().repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    y, size = x @ w.t(), x.abs() @ w.abs().t()
    err = size * (132 + K / 128 + 2) * U
    return y, err + ROUND[dtype] * (y.abs() + err) + TINY[dtype]
