"""The C entry points and the binding of the 8-bit steps around the projections: sizes and host-side
refusals (CPU only: every call here returns before it touches a device)."""
import ctypes
import os
import re

import pytest

import q6_int8_mmq_gb300 as q6
from q6_int8_mmq_gb300 import build as q6build

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: the call is refused before
ODD = ctypes.c_void_p(0x10008)
ODDEST = ctypes.c_void_p(0x10001)
BIG = 1 << 40
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    q6build.build()
    return q6.load()


def refused(rc, code):
    assert rc == code, (rc, q6.load().q6_last_error())


def test_path_names_match_the_header():
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "q6mmq.h")).read()
    defs = dict(re.findall(r"#define (Q6_\w+) (\d+)", text))
    assert int(defs["Q6_PATH_F8_FEW"]) == q6.PATH_F8_FEW and int(defs["Q6_PATH_F8_TC"]) == q6.PATH_F8_TC
    assert len(q6.PATH_NAMES) == len(set(q6.PATH_NAMES.values())) == q6.PATH_F8_TC + 1


def test_sizes(lib):
    assert q6.f8_act_bytes(5, 272) == (5 * 272, 3 * 8 * 4, 8)
    assert q6.f8_act_bytes(0, 16) == (0, 0, 0)
    assert q6.f8_act_bytes(8, 128) == (1024, 32, 8)
    assert q6.f8_weight_bytes(129, 400) == (129 * 400, 2 * 4 * 4)
    for rows, K in ((-1, 16), (1, 0), (1, 8), (1, 100), (2 ** 31 - 1, 16), (2 ** 30, 2048)):
        for call in (q6.f8_act_bytes, q6.f8_weight_bytes):
            with pytest.raises(q6.Q6Error):
                call(rows, K)
    with pytest.raises(q6.Q6Error):
        q6.f8_weight_bytes(0, 16)


def norm(lib, f8=True, X=FAKE, type=F32, ldx=512, r=FAKE, rtype=F32, ldr=512, w=FAKE, wtype=F32, eps=1e-6,
         N=3, K=512, h=FAKE, ldh=512, q=FAKE, scale=FAKE, xh=None, us=None):
    if f8:
        return lib.q6_rms_norm_f8(X, type, ldx, r, rtype, ldr, w, wtype, eps, N, K, h, ldh, q, scale, None)
    return lib.q6_rms_norm_q8(X, type, ldx, r, rtype, ldr, w, wtype, eps, N, K, h, ldh, q, scale, xh, us,
                              None)


@pytest.mark.parametrize("f8", [True, False])
def test_norm_refusals(lib, f8):
    def call(**kw):
        return norm(lib, f8, **kw)

    for kw in (dict(N=-1), dict(K=0), dict(K=520), dict(ldx=511), dict(type=3), dict(wtype=-1), dict(rtype=7),
               dict(ldr=504), dict(ldh=500), dict(X=None), dict(w=None), dict(h=None), dict(q=None),
               dict(scale=None), dict(r=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(eps=1e-40)):
        refused(call(**kw), q6.Q6_EINVAL)
    for kw in (dict(X=ODD), dict(ldx=514), dict(type=BF16, ldx=516), dict(r=ODD), dict(ldr=513), dict(h=ODD),
               dict(ldh=518, rtype=BF16), dict(w=ODD), dict(q=ODD), dict(scale=ODD)):
        refused(call(**kw), q6.Q6_EALIGN)
    refused(call(K=131072 + 256, ldx=BIG, ldr=BIG, ldh=BIG), q6.Q6_ESIZE)
    refused(call(N=2 ** 31 - 1), q6.Q6_ESIZE)
    assert call(N=0, X=None) == 0
    if not f8:
        refused(call(K=128), q6.Q6_EINVAL)
        refused(call(xh=ODD), q6.Q6_EALIGN)
        refused(call(us=ODD), q6.Q6_EALIGN)


def test_activation_and_quantiser_refusals(lib):
    def f8(X=FAKE, type=F32, N=3, K=512, ldx=1024, q=FAKE, s=FAKE):
        return lib.q6_silu_mul_f8(X, type, N, K, ldx, q, s, None)

    def q8(X=FAKE, type=F32, N=3, K=512, ldx=1024, q=FAKE, s=FAKE):
        return lib.q6_silu_mul_q8(X, type, N, K, ldx, q, s, None, None, None)

    def act(X=FAKE, type=F32, N=3, K=512, ldx=1024, q=FAKE, s=FAKE):
        return lib.q6_f8_quantize_act(X, type, N, K, ldx, q, s, None)

    def weight(X=FAKE, type=F32, N=3, K=512, ldx=1024, q=FAKE, s=FAKE):
        return lib.q6_f8_quantize_weights(X, type, N, K, ldx, q, s, None)

    for call in (f8, q8, act, weight):
        for kw in (dict(N=-1), dict(K=0), dict(K=24), dict(type=3), dict(X=None), dict(q=None), dict(s=None),
                   dict(ldx=511)):
            refused(call(**kw), q6.Q6_EINVAL)
        for kw in (dict(X=ODD), dict(ldx=1030), dict(type=BF16, ldx=1028), dict(q=ODD), dict(s=ODDEST)):
            refused(call(**kw), q6.Q6_EALIGN)
        refused(call(N=2 ** 31 - 100), q6.Q6_ESIZE)
    for call in (f8, q8):
        refused(call(ldx=1023), q6.Q6_EINVAL)
    for call in (f8, q8, act):
        assert call(N=0, X=None) == 0
        refused(call(s=ODD), q6.Q6_EALIGN)
    refused(weight(N=0), q6.Q6_EINVAL)


def test_product_refusals(lib):
    path = ctypes.c_int(9)

    def call(wq=FAKE, sw=FAKE, M=64, K=512, xq=FAKE, sx=FAKE, N=3, Y=FAKE, type=F32, ldy=64):
        return lib.q6_f8_mmq(wq, sw, M, K, xq, sx, N, Y, type, ldy, ctypes.byref(path), None)

    for kw in (dict(M=0), dict(M=-1), dict(N=-1), dict(K=0), dict(K=40), dict(type=3), dict(ldy=63),
               dict(wq=None), dict(sw=None), dict(xq=None), dict(sx=None), dict(Y=None)):
        refused(call(**kw), q6.Q6_EINVAL)
        assert path.value == q6.PATH_NONE
    for kw in (dict(wq=ODD), dict(xq=ODD), dict(sx=ODD), dict(sw=ODDEST), dict(Y=ODDEST),
               dict(Y=ODDEST, type=BF16)):
        refused(call(**kw), q6.Q6_EALIGN)
    for kw in (dict(M=2 ** 31 - 1, K=16, ldy=BIG), dict(N=2 ** 31 - 1, K=16), dict(M=2 ** 29, K=4096, ldy=BIG),
               dict(M=2 ** 30, N=2 ** 30, K=16, ldy=BIG)):
        refused(call(**kw), q6.Q6_ESIZE)
    assert call(N=0, xq=None, Y=None) == 0


def test_the_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    x, w = torch.ones(3, 512), torch.ones(512)
    e4m3 = torch.zeros(3, 512, dtype=torch.float8_e4m3fn)
    for call in (lambda: q6.f8_quantize_act(x),                       # host memory
                 lambda: q6.f8_quantize_act(x.double()),
                 lambda: q6.f8_quantize_act(x[0]),
                 lambda: q6.f8_quantize_act("x"),
                 lambda: q6.f8_quantize_weights(x),
                 lambda: q6.rms_norm_q8(x, w, 1e-6),
                 lambda: q6.rms_norm_f8(x, w, 1e-6, residual=x),
                 lambda: q6.silu_mul_q8(x),
                 lambda: q6.silu_mul_f8(x[:, :511]),
                 lambda: q6.F8Activations(3, 512, e4m3, torch.zeros(4, 3)),
                 lambda: q6.F8Activations(3, 512, e4m3, torch.zeros(4, 4)),
                 lambda: q6.F8Activations(3, 512, e4m3.view(torch.uint8), torch.zeros(4, 4)),
                 lambda: q6.F8Weights(3, 512, e4m3, torch.zeros(1, 4)),
                 lambda: q6.F8Weights(3, 512, e4m3, torch.zeros(2, 4)),
                 lambda: q6.F8Weights(0, 512, e4m3, torch.zeros(0, 4)),
                 lambda: q6.alloc_f8_activations(3, 512, "cpu"),
                 lambda: q6.alloc_f8_weights(3, 512, "cpu"),
                 lambda: q6.alloc_f8_activations(3, 100),
                 lambda: q6.alloc_f8_weights(0, 16)):
        with pytest.raises(q6.Q6Error):
            call()
