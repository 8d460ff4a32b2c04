"""Roundings of the grouped K-quant products against what they are stated to be, the persistent
walk of the tensor-core kernel over many tiles, and every pair of types of the adapters (GPU)."""
import numpy as np
import pytest

import q6_int8_mmq_gb300 as q6

import moe_reference as ref
from test_gpu_moe import TYPE, built, check, cuda, f64, rng, run_lora  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def blocks(gen, fmt, E, M, K, spread):
    """Random raw experts [E, M, bytes]: block scales spread by a factor of exp(spread * N(0, 1))."""
    raw = torch.randint(0, 256, (E, M, K // 256, ref.BLOCK[fmt]), generator=gen, dtype=torch.uint8)
    vary = torch.exp(spread * torch.randn(E, M, K // 256, 1, generator=gen)) / np.sqrt(K)
    if fmt == "q4_K":
        raw[..., 0:2] = (vary / 170).half().view(torch.uint8)
        raw[..., 2:4] = (vary * (6 + 3 * torch.rand(E, M, K // 256, 1, generator=gen)) / 170).half().view(torch.uint8)
    else:
        raw[..., 208:210] = (vary / 1370).half().view(torch.uint8)
    return raw.flatten(2)


def rounding_squares(raw, fmt, kernel, type, glu, wide=False):
    """For each weight of raw [rows, bytes] an upper bound of the expected square of the error it
    enters the sums with. A rounding to 11 bits is uniform within half a step, at most 2^-11 of the
    value: a third of that, squared. What is rounded:
      few-token kernel    q4_K nothing; q6_K sc * (q - 32), where it is above 2048
      tensor cores, bf16  q4_K sc * d (so the code's term), dmin * m and the weight; q6_K sc * d
                          and the weight
      tensor cores, f16   the weight; for q4_K its min's offset too, at most 2^-12 of sc * d. With
                          gate and up rows nothing (22 bits).
    And on the tensor cores half of the smallest binary16 step, at most 2^-34 of a row's largest
    possible weight, or 2^-19 in bf16 products of rows not marked to keep a wide range, for the min
    and the weight."""
    w = ref.dequantise(raw, fmt)
    b = raw.reshape(raw.shape[0], -1, ref.BLOCK[fmt])

    def half(at):
        return np.abs(np.ascontiguousarray(b[..., at:at + 2]).view(np.float16).astype(np.float64))[..., 0]

    one = (2.0 ** -11) ** 2 / 3
    d = half(0 if fmt == "q4_K" else 208)
    if kernel == "experts_few":
        if fmt == "q4_K":
            return np.zeros_like(w)
        return np.where(np.abs(w) > 2048 * np.repeat(d, 256, 1), one * w ** 2, 0.0)
    largest = (945 * d + 63 * half(2) if fmt == "q4_K" else 4096 * d).max(1)
    floor = 2.0 ** -34 if wide or type == "f16" else 2.0 ** -19
    sq = 2 * (floor * largest[:, None]) ** 2 / 3 + np.zeros_like(w)
    if type == "f16" and glu:
        return sq
    if fmt == "q6_K":
        return sq + (1 if type == "f16" else 2) * one * w ** 2
    no_min, full = b.copy(), b.copy()
    no_min[..., 2:4] = 0
    full[..., 2:4], full[..., 16:] = 0, 255
    code = ref.dequantise(no_min.reshape(raw.shape), fmt)
    step = ref.dequantise(full.reshape(raw.shape), fmt) / 15          # sc * d
    if type == "f16":
        return sq + one * w ** 2 + (2.0 ** -12 * step) ** 2 / 3
    return sq + one * (code ** 2 + (code - w) ** 2 + w ** 2)


def hold(rng, fmt, type, counts, M, K, swiglu, gather, spread, columns=None):
    """Runs a product over counts[e] items of expert e and holds it to the bound of every value, and
    as a whole to 1.1 times the error of one rounding of the result and the stated roundings of the
    weights (tens of thousands of values: the norms are within a few per cent of their expected
    values). Of `columns` output features; returns the path."""
    E = len(counts)
    ids = rng.permutation(np.repeat(np.arange(E), counts))[:, None]
    raw = blocks(torch.Generator().manual_seed(int(rng.integers(1 << 30))), fmt, E, M, K, spread)
    w = q6.pack_experts(raw.cuda(), fmt, E, M, K, swiglu=swiglu)
    X = cuda(rng.standard_normal((len(ids), K)), type)
    Y, path = q6.experts_mmq(w, X, q6.group_rows(cuda(ids.astype(np.int32)), E), gather=gather)
    q6.sync_status()
    out = M // 2 if swiglu else M
    cols = np.arange(out)
    if columns is not None:
        cols = np.unique(np.concatenate([[0, out - 1, out // 2], rng.integers(0, out, columns)]))
    rows = np.concatenate([cols, out + cols]) if swiglu else cols
    some = raw[:, torch.from_numpy(rows)].numpy()
    x = f64(X)
    want, bound = ref.experts(some, fmt, x, ids, E, swiglu, gather, type)
    got = f64(Y[:, torch.from_numpy(cols).cuda()])
    fits = np.full(want.shape, True)
    if type == "f16":                    # what binary16 rounds to an infinity has to be one
        fits = np.abs(want) + bound < 65520
        assert (np.isposinf(np.abs(got)) & (np.sign(got) == np.sign(want))
                | (np.abs(got - want) <= bound))[~fits].all()
        assert fits.mean() > 0.99
    check(torch.from_numpy(np.where(fits, got, 0)), np.where(fits, want, 0), bound)
    offsets, token, _ = ref.group(ids, E)
    rounded = torch.from_numpy(np.where(fits, want, 0)).to(TYPE[type]).double().numpy()
    expected = ((rounded - want)[fits] ** 2).sum()
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        xe = x[token[i]] if gather else x[i]
        var = xe ** 2 @ rounding_squares(some[e], fmt, path, type, swiglu).T
        if swiglu:
            we = ref.dequantise(some[e], fmt)
            g, u = np.split(xe @ we.T, 2, axis=1)
            s = 0.5 + 0.5 * np.tanh(g / 2)
            slope = s * (1 + g * (1 - s))                   # of g * s
            var = (slope * u) ** 2 * var[:, :len(cols)] + (g * s) ** 2 * var[:, len(cols):]
        expected += var[fits[i]].sum()
    assert np.linalg.norm((got - want)[fits]) <= 1.1 * np.sqrt(expected)
    return path


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("spread", [0.3, 2.0])     # beyond a few times 2^7 rows go another way
@pytest.mark.parametrize("path", ["experts_few", "experts_tc"])
def test_weights_are_rounded_as_stated(rng, fmt, type, swiglu, spread, path):
    counts = [1] * 50 + [0] * 14 if path == "experts_few" else [200, 130, 70]
    assert hold(rng, fmt, type, counts, 512, 1024, swiglu, True, spread) == path


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [768, 1024, 1280])
def test_many_tiles_a_pair(rng, fmt, type, swiglu, K):
    """Each pair of SMs (76 at the most) walks four to five of 342 tiles of 1 to 256 items, odd and
    even numbers of super-blocks: what a tile leaves in the rings, slots and barriers, the two
    accumulators in turn and as one, the list taken to and fro."""
    counts = [1, 5, 40, 100, 128, 129, 130, 200, 256, 257, 300, 500, 0, 33, 64, 310]
    assert hold(rng, fmt, type, counts, 4600, K, swiglu, K != 1024, 0.3, 40) == "experts_tc"


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type,swiglu", [("bf16", True), ("f16", False), ("f16", True)])
def test_many_tiles_of_many_experts(rng, fmt, type, swiglu):
    """More experts than are put in order of size."""
    counts = rng.integers(0, 5, 300)
    counts[[7, 150, 299]] = 129, 260, 150
    assert hold(rng, fmt, type, counts, 360, 768, swiglu, True, 0.3, 30) == "experts_tc"


@pytest.mark.parametrize("N,L,r,K,M", [(1, 1, 8, 32, 1), (2, 3, 24, 96, 33), (47, 24, 32, 1024, 200),
                                       (100, 2, 64, 512, 130), (333, 5, 128, 1056, 97),
                                       (40, 1, 256, 288, 64), (65, 1, 72, 64, 300)])
@pytest.mark.parametrize("xtype", ["bf16", "f16"])
def test_lora_f16_adapters_of_16_bit_x(rng, N, L, r, K, M, xtype):
    run_lora(rng, N, L, r, K, M, xtype, "f16")


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,E", [(240, 2), (40, 48)])
@pytest.mark.parametrize("step", [2, 3])
def test_super_blocks_far_apart_keep_their_bits(rng, fmt, type, swiglu, N, E, step):
    """Rows whose super-blocks differ by up to 2^21, with scales of any mantissa, and tokens that look
    at one super-block each: each super-block's results as a whole within 1.1 times the error of one
    rounding and the stated roundings of the weights (over thousands of values), whose smallest is
    half of a binary16 step or 2^-34 of the row's largest possible weight."""
    M, K = 256, 2048
    raw = blocks(torch.Generator().manual_seed(int(rng.integers(1 << 30))), fmt, E, M, K, 0.0).numpy()
    b = raw.reshape(E, M, K // 256, ref.BLOCK[fmt])
    level = 2.0 ** (6 - step * np.arange(K // 256))         # down to 2^-15

    def scales():
        return (level * rng.uniform(1, 2, b.shape[:3])).astype(np.float16)[..., None].view(np.uint8)

    at = 0 if fmt == "q4_K" else 208
    b[..., at:at + 2] = scales()
    if fmt == "q4_K":
        b[..., 2:4] = scales()
    x, mine = np.zeros((N, K)), np.arange(N) % (K // 256)
    for n in range(N):      # results of about 16, so that binary16 ones have all their bits
        x[n, 256 * mine[n]:256 * mine[n] + 256] = rng.standard_normal(256) / level[mine[n]] / 256
    X = cuda(x, type)
    x = f64(X)
    ids = rng.integers(0, E, (N, 1))
    w = q6.pack_experts(cuda(raw), fmt, E, M, K, swiglu=swiglu)
    Y, path = q6.experts_mmq(w, X, q6.group_rows(cuda(ids.astype(np.int32)), E))
    assert path == ("experts_tc" if N > E else "experts_few")
    want, _ = ref.experts(raw, fmt, x, ids, E, swiglu, True, type)
    rounded = torch.from_numpy(want).to(TYPE[type]).double().numpy()
    expected, got = (rounded - want) ** 2, f64(Y)
    fits = np.isfinite(rounded) & (np.abs(rounded) < (60000 if type == "f16" else np.inf))
    assert fits.mean() > 0.9 and np.isfinite(got[fits]).all()
    offsets, token, _ = ref.group(ids, E)
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        var = x[token[i]] ** 2 @ rounding_squares(raw[e], fmt, path, type, swiglu, True).T
        if swiglu:
            g, u = np.split(x[token[i]] @ ref.dequantise(raw[e], fmt).T, 2, axis=1)
            s = 0.5 + 0.5 * np.tanh(g / 2)
            slope = s * (1 + g * (1 - s))
            var = (slope * u) ** 2 * var[:, :M // 2] + (g * s) ** 2 * var[:, M // 2:]
        expected[i] += var
    for s in range(K // 256):
        of = (mine[token] == s)[:, None] & fits
        assert np.linalg.norm((got - want)[of]) <= 1.1 * np.sqrt(expected[of].sum()), s
