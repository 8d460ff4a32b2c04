"""The C entry points of expert routing, grouped products, combination and adapters: sizes and
host-side refusals (CPU only: every call here returns before it touches a device)."""
import ctypes

import pytest

import q6_int8_mmq_gb300 as q6
from q6_int8_mmq_gb300 import build as q6build, moe

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: the call is refused before
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    q6build.build()
    return q6.load()


def test_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "q6mmq.h")).read()
    defs = dict(re.findall(r"#define (Q6_\w+) (\d+)", text))
    assert int(defs["Q6_MAX_GROUPS"]) == moe.MAX_GROUPS
    assert int(defs["Q6_MAX_TOPK"]) == moe.MAX_TOPK
    assert int(defs["Q6_LORA_MAX_RANK"]) == moe.LORA_MAX_RANK
    assert (int(defs["Q6_FMT_Q4K"]), int(defs["Q6_FMT_Q6K"])) == (moe.FORMATS["q4_K"],
                                                                   moe.FORMATS["q6_K"])
    assert int(defs["Q6_PATH_EXPERTS_FEW"]) == q6.PATH_EXPERTS_FEW
    assert int(defs["Q6_PATH_EXPERTS_TC"]) == q6.PATH_EXPERTS_TC


def test_plane_bytes(lib):
    # tiles of 128 rows x 256 of K, and 4 bytes a row
    assert q6.expert_plane_bytes("q4_K", 1, 1, 256) == 128 * 144 + 128 * 4
    assert q6.expert_plane_bytes("q6_K", 3, 130, 512) == 3 * 2 * (2 * 128 * 210 + 128 * 4)
    # 9 gate and 9 up rows are two blocks of 16 plane rows
    assert q6.expert_plane_bytes("q4_K", 2, 18, 256, True) == 2 * (128 * 144 + 128 * 4)
    assert q6.expert_plane_bytes("q4_K", 1, 2 * 65 * 8, 256, True) == 9 * (128 * 144 + 128 * 4)


@pytest.mark.parametrize("fmt,E,M,K,glu", [("q4_K", 0, 4, 256, 0), ("q4_K", 1025, 4, 256, 0),
                                           ("q6_K", 1, 0, 256, 0), ("q6_K", 1, 4, 128, 0),
                                           ("q6_K", 1, 5, 256, 1)])
def test_plane_bytes_refuses(lib, fmt, E, M, K, glu):
    with pytest.raises(q6.Q6Error):
        moe.expert_plane_bytes.__wrapped__(fmt, E, M, K, bool(glu))


def test_workspaces(lib):
    assert q6.group_workspace_bytes(64, 8, 256) == 0              # one block does it
    assert q6.group_workspace_bytes(65, 8, 256) == 65 * 260 * 4   # a row of counts a block
    assert q6.group_workspace_bytes(100000, 8, 7) == 152 * 8 * 4
    bf16, f16 = 1, 2
    # few items: X is read as it is; many: binary16 rows, and bf16's scales
    assert moe.experts_workspace_bytes(8, 512, bf16, 8, True) == 0
    assert moe.experts_workspace_bytes(8, 512, bf16, 9, False) == -(-9 * 1024 // 256) * 256 + 9 * 4
    assert moe.experts_workspace_bytes(8, 512, f16, 9, False) == 0
    assert moe.experts_workspace_bytes(8, 512, f16, 9, True) == -(-9 * 1024 // 256) * 256
    assert q6.lora_workspace_bytes(80, 10, 16, 4096) == 0
    assert q6.lora_workspace_bytes(81, 10, 16, 4096) % (81 * 16 * 4) == 0
    assert q6.lora_workspace_bytes(81, 10, 16, 4096) > 0
    for bad in ((1, 0, 4), (1, 33, 4), (1, 1, 0), (1, 1, 1025), (-1, 1, 4), (1 << 30, 2, 4)):
        with pytest.raises(q6.Q6Error):
            moe.group_workspace_bytes.__wrapped__(*bad)
    for bad in ((1, 1, 4, 64), (1, 1, 264, 64), (1, 1, 12, 64), (1, 1, 8, 48), (1, 0, 8, 64),
                (-1, 1, 8, 64)):
        with pytest.raises(q6.Q6Error):
            moe.lora_workspace_bytes.__wrapped__(*bad)


def test_group_and_route_refusals(lib):
    def group(ids=FAKE, N=100, per=8, G=16, offsets=FAKE, rows=FAKE, pos=FAKE, ws=FAKE, n=BIG):
        return lib.q6_group_rows(ids, N, per, G, offsets, rows, pos, ws, n, None)

    assert group(ids=None) == q6.Q6_EINVAL
    assert group(offsets=None) == q6.Q6_EINVAL
    assert group(pos=None) == q6.Q6_EINVAL
    assert group(G=2000) == q6.Q6_EINVAL
    assert group(rows=ODD) == q6.Q6_EALIGN
    assert group(ws=ODD) == q6.Q6_EALIGN
    assert group(ws=None) == q6.Q6_ESIZE
    assert group(n=100 * 20 * 4 - 1) == q6.Q6_ESIZE
    assert lib.q6_last_error()

    def route(logits=FAKE, type=0, N=100, E=16, ldl=16, k=8, ids=FAKE, w=FAKE, ws=FAKE, n=BIG):
        return lib.q6_moe_route(logits, type, N, E, ldl, k, 1, ids, w, FAKE, FAKE, FAKE, ws, n, None)

    assert route(type=3) == q6.Q6_EINVAL
    assert route(ldl=15) == q6.Q6_EINVAL
    assert route(k=17) == q6.Q6_EINVAL
    assert route(logits=None) == q6.Q6_EINVAL
    assert route(w=None) == q6.Q6_EINVAL
    assert route(logits=ODD) == q6.Q6_EALIGN
    assert route(n=4) == q6.Q6_ESIZE


def test_experts_refusals(lib):
    path = ctypes.c_int(-1)

    def mmq(fmt=4, plane=FAKE, E=4, M=64, K=512, glu=0, X=FAKE, type=1, nx=100, ldx=512, gather=1,
            offsets=FAKE, rows=FAKE, items=100, Y=FAKE, ldy=64, ws=FAKE, n=BIG):
        return lib.q6_experts_mmq(fmt, plane, E, M, K, glu, X, type, nx, ldx, gather, offsets, rows,
                                  items, Y, ldy, ws, n, ctypes.byref(path), None)

    assert mmq(fmt=5) == q6.Q6_EINVAL
    assert mmq(K=300) == q6.Q6_EINVAL
    assert mmq(type=0) == q6.Q6_EINVAL                     # f32 activations
    assert mmq(ldx=504) == q6.Q6_EINVAL
    assert mmq(ldy=63) == q6.Q6_EINVAL
    assert mmq(M=63, glu=1) == q6.Q6_EINVAL
    assert mmq(gather=0, nx=99) == q6.Q6_EINVAL            # fewer rows than items
    assert mmq(rows=None) == q6.Q6_EINVAL
    assert mmq(plane=None) == q6.Q6_EINVAL
    assert mmq(X=ctypes.c_void_p(0x10008)) == q6.Q6_EALIGN
    assert mmq(ldx=516) == q6.Q6_EALIGN
    assert mmq(plane=ctypes.c_void_p(0x10010)) == q6.Q6_EALIGN
    assert mmq(items=0) == q6.Q6_OK and path.value == q6.PATH_NONE
    assert lib.q6_pack_experts(4, None, 1, 4, 256, 0, FAKE, None) == q6.Q6_EINVAL
    assert lib.q6_pack_experts(4, FAKE, 1, 4, 256, 0, ODD, None) == q6.Q6_EALIGN


def test_combine_and_lora_refusals(lib):
    def combine(Y=FAKE, type=1, ldy=64, N=3, k=2, M=64, shared=None, lds=0, out=FAKE, ldo=64):
        return lib.q6_moe_combine(Y, type, ldy, FAKE, FAKE, N, k, M, shared, lds, out, ldo, None)

    assert combine(type=0) == q6.Q6_EINVAL
    assert combine(ldy=63) == q6.Q6_EINVAL
    assert combine(shared=FAKE, lds=60) == q6.Q6_EINVAL
    assert combine(k=33) == q6.Q6_EINVAL
    assert combine(out=None) == q6.Q6_EINVAL
    assert combine(out=ctypes.c_void_p(0x10001)) == q6.Q6_EALIGN
    assert combine(N=0) == q6.Q6_OK

    def lora(A=FAKE, type=1, L=2, r=16, M=64, K=512, X=FAKE, xtype=0, ldx=512, items=100, Y=FAKE,
             ldy=64, out=FAKE, ldo=64, ws=FAKE, n=BIG):
        return lib.q6_lora_add(A, FAKE, FAKE, type, L, r, M, K, X, xtype, ldx, FAKE, FAKE, items, Y,
                               ldy, out, ldo, ws, n, None)

    assert lora(type=0) == q6.Q6_EINVAL
    assert lora(xtype=3) == q6.Q6_EINVAL
    assert lora(r=12) == q6.Q6_EINVAL
    assert lora(ldx=500) == q6.Q6_EINVAL
    assert lora(ldy=60) == q6.Q6_EINVAL
    assert lora(Y=None) == q6.Q6_EINVAL
    assert lora(A=ctypes.c_void_p(0x10008)) == q6.Q6_EALIGN
    assert lora(ldx=513) == q6.Q6_EALIGN
    assert lora(out=ODD) == q6.Q6_EALIGN
    assert lora(ws=None) == q6.Q6_ESIZE
    assert lora(items=0) == q6.Q6_OK


def test_binding_refuses_what_is_no_tensor():
    for call in (lambda: q6.moe_route([[1.0]], 1), lambda: q6.group_rows([1], 1),
                 lambda: q6.pack_experts(b"", "q4_K", 1, 1, 256),
                 lambda: q6.expert_plane_bytes("q5_K", 1, 1, 256)):
        with pytest.raises(q6.Q6Error):
            call()
