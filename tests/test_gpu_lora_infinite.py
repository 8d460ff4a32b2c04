"""Infinite and NaN activations of the adapters: each gives what its products give, whichever kernels
run, and no other token sees them (GPU)."""
import numpy as np
import pytest

import q6_int8_mmq_gb300 as q6

from test_gpu_moe import built, cuda, f64, rng  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def same(got, want):
    """Equal infinities, and NaN where NaN is."""
    return np.isnan(got) & np.isnan(want) | (got == want)


@pytest.mark.parametrize("xtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("r", [8, 64])
@pytest.mark.parametrize("N", [1, 6, 40, 200])
def test_infinite_activations_of_adapters(rng, xtype, type, r, N):
    """With positive A and B an infinite x makes infinities of its sign, with an A of 0 NaN."""
    L, K, M = 2, 288, 70
    A = cuda(rng.uniform(0.1, 1, (L, r, K)) / K, type)
    B = cuda(rng.uniform(0.1, 1, (L, M, r)), type)
    X, Y = cuda(rng.standard_normal((N, K)), xtype), cuda(rng.standard_normal((N, M)), "f32")
    ids = np.arange(N) % L
    ad = q6.LoraAdapters(A, B, torch.ones(L, device="cuda"))
    g = q6.group_rows(cuda(ids.astype(np.int32)), L)
    good = q6.lora_add(ad, X, g, Y, out=torch.empty_like(Y))
    hit = {0: float("inf")} if N == 1 else {0: float("inf"), 3: -float("inf"), 4: float("nan")}
    for n, v in hit.items():
        X[n, 5 + 40 * n] = v
    out = q6.lora_add(ad, X, g, Y, out=torch.empty_like(Y))
    for n, v in hit.items():
        assert same(f64(out[n]), np.full(M, v)).all(), (n, v, out[n, :4])
    rest = [n for n in range(N) if n not in hit]
    assert torch.equal(out[rest], good[rest])
    A[:, r - 1, 5] = 0
    out = q6.lora_add(ad, X, g, Y, out=torch.empty_like(Y))
    assert torch.isnan(out[0]).all()


@pytest.mark.parametrize("N", [2, 100])
@pytest.mark.parametrize("bits", [0x7F800001, 0xFFBFFFFF, 0x7FC00000])
def test_every_nan_of_f32_stays_one(rng, N, bits):
    """Also those whose upper half alone would be an infinity."""
    A, B = cuda(rng.uniform(0.1, 1, (1, 8, 64)), "bf16"), cuda(rng.uniform(0.1, 1, (1, 33, 8)), "bf16")
    X, Y = cuda(rng.standard_normal((N, 64)), "f32"), torch.zeros((N, 33), device="cuda")
    X.view(torch.int32)[1, 20] = int(np.uint32(bits).astype(np.int32))
    for type in ("bf16", "f16"):
        ad = q6.LoraAdapters(A.to(getattr(torch, {"bf16": "bfloat16", "f16": "float16"}[type])),
                             B.to(getattr(torch, {"bf16": "bfloat16", "f16": "float16"}[type])),
                             torch.ones(1, device="cuda"))
        out = q6.lora_add(ad, X, q6.group_rows(torch.zeros(N, dtype=torch.int32, device="cuda"), 1),
                          Y, out=torch.empty_like(Y))
        assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()
