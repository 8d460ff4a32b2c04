"""The combination of very wide rows (GPU)."""
import pytest

import q6_int8_mmq_gb300 as q6

from test_gpu_moe import built  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("M", [65535 * 128, 65535 * 128 + 3, 65535 * 1024 + 8])
def test_combine_of_more_columns_than_a_grid_has_blocks(M):
    """A grid has 65535 blocks for the columns, of 128 (at widths that are no multiple of 8) or 1024."""
    Y = torch.arange(3 * M, device="cuda", dtype=torch.int32).remainder_(251).bfloat16().view(3, M)
    pos = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, 0.25], [2.0, 1.0]], device="cuda")
    shared = torch.ones((2, M), device="cuda")
    out = q6.moe_combine(Y, pos, weights, shared=shared)
    assert torch.equal(out[0], (1 + 0.5 * Y[2].float() + 0.25 * Y[0].float()).bfloat16())
    assert torch.equal(out[1], (1 + 2.0 * Y[1].float()).bfloat16())
