"""Infinite and NaN activations: each gives what its products with the weights give, whichever
kernel runs, and no other token sees them (GPU)."""
import numpy as np
import pytest

import q6_int8_mmq_gb300 as q6

import moe_reference as ref
from test_gpu_moe import built, cuda, f64, raw_experts, rng  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def same(got, want):
    """Equal infinities, and NaN where NaN is."""
    return np.isnan(got) & np.isnan(want) | (got == want)


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("N,E", [(3, 8), (5, 5), (24, 30), (300, 2)])
@pytest.mark.parametrize("M,K,gather", [(40, 512, True), (150, 7936, False)])
def test_infinite_activations_of_experts(rng, fmt, type, N, E, M, K, gather):
    """A weight of 0 makes NaN of an infinity, every other weight an infinity of its sign; of more
    than one infinity the sum counts. (The tensor-core kernel's weights have 11 bits of their terms:
    those below 2^-9 of a row's largest may come out 0.)"""
    raw = raw_experts(4, fmt, E, M, K)
    raw.reshape(E, M, -1, ref.BLOCK[fmt])[:, 3, :, :16] = 0          # a row with weights of 0
    if fmt == "q6_K":
        raw.reshape(E, M, -1, ref.BLOCK[fmt])[:, 3, :, 192:200] = 0
    ids = np.full((N, 1), 1)
    w = q6.pack_experts(cuda(raw), fmt, E, M, K)
    g = q6.group_rows(cuda(ids.astype(np.int32)), E)
    X = cuda(rng.standard_normal((N, K)), type)
    good = q6.experts_mmq(w, X, g, gather=gather)[0].clone()
    inf = float("inf")
    X[0, 7], X[1, K - 5] = inf, -inf
    X[2, 300], X[2, 5] = inf, -inf
    if N > 3:
        X[3, 100:103] = inf
        X[4, K - 256] = float("nan")
    hit = min(N, 5)
    Y, path = q6.experts_mmq(w, X, g, gather=gather)
    q6.sync_status()
    assert path == ("experts_tc" if N > E else "experts_few")
    assert torch.equal(Y[hit:], good[hit:])
    weights = ref.dequantise(raw[1], fmt)
    x, got = f64(X[:hit]), f64(Y[:hit])
    with np.errstate(invalid="ignore"):
        want = np.stack([sum(row[k] * weights[:, k] for k in np.flatnonzero(~np.isfinite(row)))
                         for row in x])
    ok = same(got, want)
    if path == "experts_tc":
        small = np.abs(weights) < 2.0 ** -9 * np.abs(weights).max(1, keepdims=True)
        unsure = np.stack([small[:, ~np.isfinite(row)].any(1) for row in x])
        assert unsure.mean() < 0.5
        ok |= unsure & ~np.isfinite(got)
    assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])


@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
def test_infinite_activations_of_gate_and_up(rng, fmt, type):
    E, H, K = 12, 20, 768
    raw = raw_experts(6, fmt, E, 2 * H, K)
    w = q6.pack_experts(cuda(raw), fmt, E, 2 * H, K, swiglu=True)
    X = cuda(rng.standard_normal((3, K)), type)
    X[0, 9], X[2, 700] = float("inf"), -float("inf")
    Y, path = q6.experts_mmq(w, X, q6.group_rows(cuda(np.full((3, 1), 5, np.int32)), E))
    assert path == "experts_few"
    weights = ref.dequantise(raw[5], fmt)
    for n, k in ((0, 9), (2, 700)):
        with np.errstate(invalid="ignore", over="ignore"):
            g, u = np.split(f64(X)[n, k] * weights[:, k], 2)
            want = g / (1 + np.exp(-g)) * u
        assert same(f64(Y)[n], want).all()
    assert torch.isfinite(Y[1]).all()
