"""Sizes of experts and adapters near the limits of the kernels' index arithmetic (CPU only: every
call here returns before it touches a device)."""
import ctypes

import pytest

import q6_int8_mmq_gb300 as q6
from q6_int8_mmq_gb300 import build as q6build, moe

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: the call is refused before
BIG = 1 << 40
MAX_ROWS = 2 ** 31 - 256             # plane rows of an expert


@pytest.fixture(scope="module")
def lib():
    q6build.build()
    return q6.load()


@pytest.mark.parametrize("M,glu", [(2 ** 31 - 1, 0), (MAX_ROWS + 1, 0), (2 ** 31 - 2, 1),
                                   (MAX_ROWS + 2, 1)])
def test_experts_of_too_many_rows_are_refused(lib, M, glu):
    """In 31 bits their bands would come out negative, and their plane small."""
    nbytes = ctypes.c_size_t()
    for fmt in (4, 6):
        assert lib.q6_expert_plane_bytes(fmt, 1, M, 256, glu, ctypes.byref(nbytes)) == q6.Q6_ESIZE
        assert lib.q6_pack_experts(fmt, FAKE, 1, M, 256, glu, FAKE, None) == q6.Q6_ESIZE
        assert lib.q6_experts_mmq(fmt, FAKE, 1, M, 256, glu, FAKE, 1, 4, 256, 1, FAKE, FAKE, 4, FAKE,
                                  1 << 31, FAKE, BIG, None, None) == q6.Q6_ESIZE
    with pytest.raises(q6.Q6Error):
        moe.expert_plane_bytes.__wrapped__("q4_K", 1, M, 256, bool(glu))


def test_the_most_rows_have_the_plane_they_need(lib):
    bands = MAX_ROWS // 128
    assert moe.expert_plane_bytes("q4_K", 1, MAX_ROWS, 256) == bands * (128 * 144 + 128 * 4)
    assert moe.expert_plane_bytes("q6_K", 1, MAX_ROWS, 256, True) == bands * (128 * 210 + 128 * 4)


@pytest.mark.parametrize("items", [1 << 31, 1 << 62, -1])
@pytest.mark.parametrize("K", [256, 1 << 20])
def test_workspace_of_too_many_items_is_refused(lib, items, K):
    """As in the product itself; 2^62 items' bytes would not fit 64 bits."""
    nbytes = ctypes.c_size_t()
    for type in (1, 2):
        assert lib.q6_experts_workspace_bytes(4, K, type, items, 1, ctypes.byref(nbytes)) == q6.Q6_EINVAL
    assert lib.q6_experts_workspace_bytes(4, K, 1, (1 << 31) - 1, 1, ctypes.byref(nbytes)) == q6.Q6_OK
    assert nbytes.value >= ((1 << 31) - 1) * (2 * K + 4)


def test_adapters_of_too_many_columns_or_items_are_refused(lib):
    """Column and tile numbers run up to a step past the last, and would leave 31 bits there."""
    nbytes = ctypes.c_size_t()

    def size(items, K):
        return lib.q6_lora_workspace_bytes(items, 2, 8, K, ctypes.byref(nbytes))

    def add(items=100, M=64, K=512):
        ld = max(M, K)
        return lib.q6_lora_add(FAKE, FAKE, FAKE, 1, 2, 8, M, K, FAKE, 1, ld, FAKE, FAKE, items, FAKE,
                               ld, FAKE, ld, FAKE, BIG, None)

    assert size(2 ** 31 - 256, 2 ** 30) == q6.Q6_OK
    assert size(100, 2 ** 31 - 32) == q6.Q6_ESIZE
    assert size(2 ** 31 - 255, 64) == q6.Q6_ESIZE
    assert add(M=2 ** 31 - 1) == q6.Q6_ESIZE
    assert add(M=2 ** 30 + 1) == q6.Q6_ESIZE
    assert add(K=2 ** 31 - 32) == q6.Q6_ESIZE
    assert add(items=2 ** 31 - 1) == q6.Q6_ESIZE
