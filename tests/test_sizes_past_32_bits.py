"""Sizes that the C ABI's 32-bit integers cannot hold are refused, not cut to their low bits. (CPU
only, but for the last test: 2^32 + 16 is 16 in 32 bits, a size that every call takes.)"""
import pytest

import q6_int8_mmq_gb300 as q6
from q6_int8_mmq_gb300 import build as q6build

WRAPS = (2 ** 32 + 256, 2 ** 33 + 256, 2 ** 31, -2 ** 32 + 256)


@pytest.fixture(scope="module", autouse=True)
def built():
    q6build.build()


@pytest.mark.parametrize("size", ["f8_act_bytes", "f8_weight_bytes", "act_plane_bytes", "act_sums_bytes",
                                  "plane_bytes", "q4k_plane_bytes"])
@pytest.mark.parametrize("n", WRAPS)
def test_sizes_that_wrap_are_refused(size, n):
    for args in ((n, 256), (3, n)):
        with pytest.raises(q6.Q6Error) as e:
            getattr(q6, size)(*args)
        assert e.value.code == q6.Q6_ESIZE
    getattr(q6, size)(256, 256)


def test_buffers_of_sizes_that_wrap_are_refused():
    pytest.importorskip("torch")
    for n in WRAPS:
        for call in (lambda: q6.alloc_f8_activations(n, 256), lambda: q6.alloc_f8_activations(3, n),
                     lambda: q6.alloc_f8_weights(n, 256), lambda: q6.alloc_f8_weights(3, n),
                     lambda: q6.alloc_activations(n, 256), lambda: q6.alloc_activations(3, n),
                     lambda: q6.F8Activations(n, 256, None, None), lambda: q6.F8Weights(n, 256, None, None),
                     lambda: q6.Activations(n, 256, None, None, None, 256)):
            with pytest.raises(q6.Q6Error):
                call()


@pytest.mark.gpu
def test_rows_of_a_length_that_wraps_are_refused():
    import torch
    K = 2 ** 32 + 256                        # 256 in 32 bits
    x = torch.empty(1, K, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(K, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: q6.f8_quantize_act(x), lambda: q6.f8_quantize_weights(x),
                 lambda: q6.silu_mul_f8(torch.empty(1, 2 * K, dtype=torch.bfloat16, device="cuda")),
                 lambda: q6.rms_norm_f8(x, w, 1e-6), lambda: q6.rms_norm_q8(x, w, 1e-6)):
        with pytest.raises(q6.Q6Error):
            call()
