"""GPU tests of the 8-bit steps around the projections: the norm and the gated activation that end
in quantised activations, the e4m3 quantisers and the product of e4m3 blocks."""
import pytest

torch = pytest.importorskip("torch")

import q6_int8_mmq_gb300 as q6  # noqa: E402
import f8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def activations(g, N, K, dtype):
    """N(0, 1) with wide channels, rows of other sizes, an all-zero row and zero blocks."""
    x = randn(g, N, K) * torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 20.0, 1.0)
    x = x * torch.exp(randn(g, N, 1))
    if N > 2:
        x[1] = 0
        x[2, :min(K, 160)] = 0
    return x.to(dtype)


def strided(t, pad):
    """The same values in rows `pad` elements further apart; what lies between must not matter."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def check_q8(act, N, t, rel, root=1.0, root_rel=0.0):
    codes = act.xh.double() if act.xh is not None else act.xq.double()
    if act.xh is not None and act.xq is not None:
        assert torch.equal(act.xh, act.xq.half())
    da = act.da[:, :N].t().double()
    ref.check_codes(codes, da, t, rel, root, root_rel, f8=False)
    if act.us is not None:      # da * (sum of the block's codes) as hi and lo parts
        K = act.K
        pairs = act.us.double()
        got = pairs.unflatten(1, (-1, 2, 8))[:, :K // 256].sum(2).flatten(1)
        want = act.da[:, :N].t().double() * codes.unflatten(1, (-1, 32)).sum(2)
        assert ((got - want).abs() <= ref.U * want.abs()).all()
        if K // 256 % 2:
            assert not pairs[:, -16:].any()


def check_f8(act, N, t, rel, root=1.0, root_rel=0.0):
    ref.check_codes(act.xq.double(), act.sx[:, :N].t().double(), t, rel, root, root_rel, f8=True)


# ------------------------------------------------------------------- norm ---

@pytest.mark.parametrize("type,rtype", [(t, r) for t in TYPES for r in (None, *TYPES)])
@pytest.mark.parametrize("N,K", [(1, 256), (3, 512), (5, 2560), (130, 768), (33, 16384)])
def test_norm_q8(N, K, type, rtype):
    g = gen(N * K)
    x = strided(activations(g, N, K, type), 8)
    r = None if rtype is None else strided((2 * activations(g, N, K, F32)).to(rtype), 16)
    w = (1 + 0.3 * randn(g, K)).to(TYPES[K // 256 % 3])
    eps = 1e-5
    h, t, root, rel, root_rel = ref.norm(x, r, w, eps)
    us = K <= 2560
    before = None if r is None else r.clone()
    act, got = q6.rms_norm_q8(x, w, eps, residual=r, h=None if r is None else torch.empty_like(r),
                              want_us=us)
    check_q8(act, N, t, rel, root, root_rel)
    if r is None:
        assert got is x
    else:
        assert torch.equal(r, before)
        bound = (ref.ROUND[rtype] + 2 * ref.U) * h.abs() + ref.TINY[rtype]
        assert ((got.double() - h).abs() <= bound).all()
        again, same = q6.rms_norm_q8(x, w, eps, residual=r, want_us=us)     # in place
        assert same is r and torch.equal(r, got)
        assert torch.equal(again.xq, act.xq) and torch.equal(again.da[:, :N], act.da[:, :N])


@pytest.mark.parametrize("type,rtype", [(t, r) for t in TYPES for r in (None, *TYPES)])
@pytest.mark.parametrize("N,K", [(1, 16), (1, 4096), (4, 112), (3, 144), (67, 1040), (9, 33008)])
def test_norm_f8(N, K, type, rtype):
    g = gen(N * K + 1)
    x = strided(activations(g, N, K, type), 16)
    r = None if rtype is None else (2 * activations(g, N, K, F32)).to(rtype)
    w = (1 + 0.3 * randn(g, K)).to(TYPES[N % 3])
    h, t, root, rel, root_rel = ref.norm(x, r, w, 1e-6)
    act, got = q6.rms_norm_f8(x, w, 1e-6, residual=r, h=None if r is None else torch.empty_like(r))
    check_f8(act, N, t, rel, root, root_rel)
    if r is not None:
        bound = (ref.ROUND[rtype] + 2 * ref.U) * h.abs() + ref.TINY[rtype]
        assert ((got.double() - h).abs() <= bound).all()


def test_norm_of_the_widest_rows():
    g = gen(1)
    K = 131072
    x, w = randn(g, 2, K), 1 + 0.1 * randn(g, K)
    h, t, root, rel, root_rel = ref.norm(x, None, w, 1e-6)
    act, _ = q6.rms_norm_q8(x, w, 1e-6, want_us=True)
    check_q8(act, 2, t, rel, root, root_rel)
    act, _ = q6.rms_norm_f8(x, w, 1e-6)
    check_f8(act, 2, t, rel, root, root_rel)


@pytest.mark.parametrize("f8", [False, True])
def test_norm_of_zeros_and_of_values_that_are_not_finite(f8):
    x = torch.ones(5, 512, device="cuda")
    x[0] = 0
    x[1, 300] = float("inf")
    x[2, 300] = float("nan")
    x[3] = 3e19              # the sum of squares is above f32's range
    w = torch.ones(512, device="cuda")
    act, _ = (q6.rms_norm_f8 if f8 else q6.rms_norm_q8)(x, w, 1e-6)
    scale = (act.sx if f8 else act.da)[:, :5].t()
    codes = act.xq.float()
    assert not codes[0].any() and not scale[0].any()
    b = 300 // (128 if f8 else 32)
    others = torch.arange(scale.shape[1], device="cuda") != b
    assert scale[1, b].isnan() and not scale[1, others].any()
    assert scale[2].isnan().all() and not codes[2].isnan().any()
    assert not scale[3].any()
    one = 448.0 if f8 else 127.0
    # 1 / (sqrt(1 + 1e-6) one): four roundings
    assert ((scale[4].double() * one * (1 + 1e-6) ** 0.5 - 1).abs() <= 4 * ref.U).all()
    assert (codes[4] == one).all()


# ------------------------------------------------------- gated activation ---

@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("N,K", [(1, 256), (3, 512), (131, 1280)])
def test_silu_q8(N, K, type):
    x = strided(activations(gen(N + K), N, 2 * K, type), 8)
    t, rel = ref.silu_mul(x)
    for xh, xq, us in ((True, True, True), (False, True, False), (True, False, False)):
        check_q8(q6.silu_mul_q8(x, want_xh=xh, want_xq=xq, want_us=us), N, t, rel)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("N,K", [(1, 16), (2, 144), (3, 528), (131, 1280)])
def test_silu_f8(N, K, type):
    x = activations(gen(N + K), N, 2 * K, type)
    t, rel = ref.silu_mul(x)
    check_f8(q6.silu_mul_f8(x), N, t, rel)


def test_silu_of_large_gates():
    """exp(-gate) above f32's range gives 0, far positive gates give gate * up."""
    x = torch.zeros(1, 512, device="cuda")
    x[0, :256] = torch.linspace(-200, 200, 256)
    x[0, 256:] = 1
    act = q6.silu_mul_q8(x)
    y = act.xq.double() * act.da[:, :1].t().repeat_interleave(32, 1).double()
    want = x[:, :256].double() * torch.sigmoid(x[:, :256].double())
    step = act.da[:, :1].t().repeat_interleave(32, 1).double()
    assert ((y - want).abs() <= 0.5001 * step + 1e-37).all()


# --------------------------------------------------------------- quantise ---

@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("N,K", [(1, 16), (3, 128), (2, 4112), (257, 1040)])
def test_quantise_act(N, K, type):
    x = strided(activations(gen(N + K), N, K, type), 24)
    check_f8(q6.f8_quantize_act(x), N, x.double(), 0.0)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (127, 128), (128, 144), (300, 1040), (129, 4096)])
def test_quantise_weights(M, K, type):
    g = gen(M + K)
    W = (randn(g, M, K) * torch.exp(randn(g, M, 1))).to(type)
    if M > 128:
        W[128:] = 0
    W = strided(W, 8)
    w = q6.f8_quantize_weights(W)
    ref.check_codes(w.wq.double(), w.sw.double(), W.double(), 0.0, 1.0, 0.0, f8=True, rows=128)


def test_quantise_of_values_that_are_not_finite_and_of_the_smallest():
    x = torch.ones(2, 512, device="cuda")
    x[0, 5] = float("nan")
    x[0, 130] = -float("inf")
    x[0, 256:384] = 2.0 ** -101
    x[1, :128] = 2.0 ** -100
    act = q6.f8_quantize_act(x)
    assert act.sx[:2, 0].isnan().all() and not act.xq[0, :384].float().any() and act.sx[2, 0] == 0
    assert act.sx[0, 1] > 0 and (act.xq[1].float() == 448).all()
    w = q6.f8_quantize_weights(x)
    assert w.sw[0, :2].isnan().all() and not w.wq[:, :256].float().any()
    assert (w.wq[:, 384:].float() == 448).all()
    assert (w.wq[1, 256:384].float() == 448).all() and not w.wq[0, 256:384].float().any()


@pytest.mark.parametrize("f8", [False, True])
def test_norm_of_many_wide_rows(f8):
    """More rows than one a SM, each longer than its CTA reads at a time."""
    g = gen(7)
    N, K = 160, 66560
    x, r = activations(g, N, K, BF16), activations(g, N, K, F32)
    w = 1 + 0.3 * randn(g, K)
    h, t, root, rel, root_rel = ref.norm(x, r, w, 1e-6)
    if f8:
        act, got = q6.rms_norm_f8(x, w, 1e-6, residual=r)
        check_f8(act, N, t, rel, root, root_rel)
    else:
        act, got = q6.rms_norm_q8(x, w, 1e-6, residual=r, want_us=True)
        check_q8(act, N, t, rel, root, root_rel)
    assert ((got.double() - h).abs() <= 2 * ref.U * h.abs()).all()


def test_of_no_rows():
    w = torch.ones(512, device="cuda")
    for dtype in TYPES:
        x = torch.empty(0, 512, dtype=dtype, device="cuda")
        assert q6.f8_quantize_act(x).xq.shape == (0, 512)
        assert q6.rms_norm_f8(x, w, 1e-6, residual=x)[0].xq.shape == (0, 512)
        assert q6.rms_norm_q8(x, w, 1e-6)[0].xq.shape == (0, 512)
        assert q6.silu_mul_f8(x).xq.shape == (0, 256) and q6.silu_mul_q8(x).xh.shape == (0, 256)
    q6.sync_status()


def test_any_sizes():
    """Forty random sizes through a chain of calls: the same checks as above."""
    import random
    rng = random.Random(11)
    for i in range(40):
        g = gen(1000 + i)
        N = int(round(2 ** rng.uniform(0, 10.5)))
        M, K = int(round(2 ** rng.uniform(0, 11.5))), 16 * int(round(2 ** rng.uniform(0, 7.5)))
        dtype = TYPES[i % 3]
        x, r = activations(g, N, K, dtype), activations(g, N, K, TYPES[i // 3 % 3])
        weight = (1 + 0.3 * randn(g, K)).to(TYPES[i // 9 % 3])
        h, t, root, rel, root_rel = ref.norm(x, r, weight, 1e-5)
        act, _ = q6.rms_norm_f8(x, weight, 1e-5, residual=r)
        check_f8(act, N, t, rel, root, root_rel)
        w = q6.f8_quantize_weights((randn(g, 2 * M, K) * torch.exp(randn(g, 2 * M, 1))).to(dtype))
        Y, _ = check_product(w, act, TYPES[(i + 1) % 3] if TYPES[(i + 1) % 3] is not F16 else BF16)
        if M % 16 == 0:
            t, rel = ref.silu_mul(Y)
            check_f8(q6.silu_mul_f8(Y), N, t, rel)


def test_scales_past_the_last_token_are_left():
    x = torch.ones(5, 256, device="cuda")
    f8, q8 = q6.alloc_f8_activations(5, 256), q6.alloc_activations(5, 256)
    for act, scale, calls in (
            (f8, f8.sx, (lambda: q6.f8_quantize_act(x, out=f8), lambda: q6.silu_mul_f8(x.repeat(1, 2), out=f8),
                         lambda: q6.rms_norm_f8(x, x[0], 1e-6, out=f8))),
            (q8, q8.da, (lambda: q6.silu_mul_q8(x.repeat(1, 2), out=q8),
                         lambda: q6.rms_norm_q8(x, x[0], 1e-6, out=q8)))):
        for call in calls:
            scale.fill_(77.0)
            call()
            assert (scale[:, 5:] == 77).all() and (scale[:, :5] != 77).all()


# ---------------------------------------------------------------- product ---

def operands(g, N, M, K):
    x, w = activations(g, N, K, F32), randn(g, M, K) * torch.exp(randn(g, M, 1))
    return q6.f8_quantize_weights(w), q6.f8_quantize_act(x)


def check_product(w, act, dtype, **more):
    Y, path = q6.f8_mmq(w, act, dtype=dtype, **more)
    q6.sync_status()
    want, bound = ref.product(act.xq, act.sx, w.wq, w.sw, dtype)
    off = (Y.double() - want).abs()
    fine = off <= bound
    if dtype is F16:
        # 65520 lies halfway between the largest binary16 value, 65504, and the next step, 65536: from
        # there on a sum rounds to infinity
        inf = Y == torch.where(want > 0, float("inf"), -float("inf"))
        fine = torch.where(want.abs() + bound >= 65520, inf | fine, fine)
        fine = torch.where(want.abs() - bound >= 65520, inf, fine)
    assert fine.all(), (path, float((off - bound)[~fine].max()))
    return Y, path


# every count of tokens at which the form of the kernel may change, and ends inside a tile
TOKENS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 192,
          193, 255, 256, 257, 383, 511, 513]


@pytest.mark.parametrize("N", TOKENS)
@pytest.mark.parametrize("M,K", [(300, 1040), (129, 400)])
def test_product_tokens(N, M, K):
    w, act = operands(gen(N), N, M, K)
    check_product(w, act, TYPES[N % 3])


@pytest.mark.parametrize("M", [1, 7, 64, 127, 128, 129, 255, 256, 257, 1000, 2056])
@pytest.mark.parametrize("N", [1, 5, 40, 130])
def test_product_rows(N, M):
    w, act = operands(gen(M), N, M, 528)
    check_product(w, act, TYPES[M % 3])


@pytest.mark.parametrize("K", [16, 32, 96, 112, 128, 144, 256, 272, 1152, 4112, 11008])
@pytest.mark.parametrize("N", [1, 3, 20, 150])
def test_product_depth(N, K):
    w, act = operands(gen(K), N, 200, K)
    check_product(w, act, TYPES[K // 16 % 3])


@pytest.mark.parametrize("N,M,K", [(1, 4096, 4096), (1, 11008, 4096), (33, 4096, 11008), (1023, 2056, 3600),
                                   (2048, 4096, 4096), (3314, 11008, 4096), (4000, 512, 3584)])
def test_product_at_size(N, M, K):
    w, act = operands(gen(N + M), N, M, K)
    check_product(w, act, BF16)


@pytest.mark.parametrize("N", [1, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("M,K", [(19585, 1040), (40000, 2064)])
def test_product_of_more_rows_than_all_sms_take_at_once(N, M, K):
    w, act = operands(gen(N + K), N, M, K)
    check_product(w, act, TYPES[N % 3])


# Few tiles and a long K: pairs of CTAs that share a tile, each with a part of K.
@pytest.mark.parametrize("K", [2176, 2304, 2448, 3568, 3600, 11008])
@pytest.mark.parametrize("N,M", [(65, 1), (129, 129), (257, 1000), (300, 70), (200, 2056), (65, 4608), (130, 4700)])
def test_product_of_few_tiles_and_a_long_k(N, M, K):
    w, act = operands(gen(N + K), N, M, K)
    check_product(w, act, TYPES[(N + K // 16) % 3])


@pytest.mark.parametrize("N,M,K", [(70, 640, 2560), (300, 1000, 3600), (130, 2056, 3600)])
def test_few_tiles_of_whole_numbers_are_exact(N, M, K):
    test_product_of_whole_numbers_is_exact(N, M, K)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [200, 2056])
def test_few_tiles_into_rows_of_a_larger_matrix(M, dtype):
    """Every alignment of Y and its rows, nothing written beside it, the same bits each time."""
    N = 140
    w, act = operands(gen(M), N, M, 3600)
    want, _ = check_product(w, act, dtype)
    for ld, at in ((M, 0), (M + 1, 0), (M + 8, 8), (M + 16, 3), (M + 3, 1)):
        big = torch.full(((N + 2) * ld + 8,), 7.0, dtype=dtype, device="cuda")
        Y = torch.as_strided(big, (N, M), (ld, 1), ld + at)
        for _ in range(4):
            got, _ = q6.f8_mmq(w, act, out=Y)
            assert torch.equal(got, want)
            Y.fill_(7.0)
        assert (big == 7).all()


@pytest.mark.parametrize("N,M,K", [(1, 640, 1024), (6, 300, 2048), (24, 513, 1024), (130, 300, 768), (700, 1025, 528)])
def test_product_of_whole_numbers_is_exact(N, M, K):
    """Codes -4 .. 4 and scales that are powers of two: every sum fits f32."""
    g = gen(N)
    small = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    power = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g, device="cuda").float())  # noqa: E731
    act = q6.F8Activations(N, K, small(N, K).to(torch.float8_e4m3fn),
                           power(-(-K // 128), -(-N // 4) * 4))
    w = q6.F8Weights(M, K, small(M, K).to(torch.float8_e4m3fn), power(-(-M // 128), -(-K // 128)))
    want, _ = ref.product(act.xq, act.sx, w.wq, w.sw, F32)
    Y, _ = q6.f8_mmq(w, act, dtype=F32)
    assert torch.equal(Y.double(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 6, 30, 140, 300])
def test_product_into_rows_of_a_larger_matrix(N, dtype):
    """Every alignment of Y and its rows, and nothing written beside it."""
    w, act = operands(gen(N), N, 200, 272)
    want, _ = check_product(w, act, dtype)
    for ld, at in ((200, 0), (201, 0), (208, 8), (216, 3), (203, 1)):
        big = torch.full(((N + 2) * ld + 8,), 7.0, dtype=dtype, device="cuda")
        Y = torch.as_strided(big, (N, 200), (ld, 1), ld + at)
        got, _ = q6.f8_mmq(w, act, out=Y)
        assert torch.equal(got, want)
        Y.fill_(7.0)
        assert (big == 7).all()


def test_product_of_nothing_and_of_nan():
    w, act = operands(gen(3), 5, 200, 272)
    Y, path = q6.f8_mmq(w, q6.alloc_f8_activations(0, 272))
    assert Y.shape == (0, 200) and path == "none"
    want, _ = q6.f8_mmq(w, act, dtype=F32)
    act.sx[1, 2] = float("nan")      # one token's second block
    Y, _ = q6.f8_mmq(w, act, dtype=F32)
    rest = [0, 1, 3, 4]
    assert Y[2].isnan().all() and torch.equal(Y[rest], want[rest])
    w.sw[1, 0] = float("inf")        # the rows from 128 on
    Y, _ = q6.f8_mmq(w, act, dtype=F32)
    assert torch.equal(Y[rest, :128], want[rest, :128]) and not Y[rest, 128:].isfinite().any()
    codes = act.xq.view(torch.uint8)
    codes[0, 3] = 0x7F               # NaN
    Y, _ = q6.f8_mmq(w, act, dtype=F32)
    assert Y[0].isnan().all() and torch.equal(Y[3, :128], want[3, :128])


def test_product_of_the_largest_codes():
    """448 * 448 in every place: no sum overflows on the way to f32."""
    for N in (1, 40, 300):
        act = q6.F8Activations(N, 512, torch.full((N, 512), 448.0, device="cuda").to(torch.float8_e4m3fn),
                               torch.ones(4, -(-N // 4) * 4, device="cuda"))
        w = q6.F8Weights(130, 512, torch.full((130, 512), 448.0, device="cuda").to(torch.float8_e4m3fn),
                         torch.ones(2, 4, device="cuda"))
        Y, _ = q6.f8_mmq(w, act, dtype=F32)
        assert (Y == 512 * 448 * 448).all()
        Y, _ = q6.f8_mmq(w, act, dtype=F16)
        assert (Y == float("inf")).all()


def test_rows_do_not_depend_on_the_batch_they_are_in():
    """The same kernel gives a token the same result whatever the others hold."""
    for N in (4, 30, 200, 600):
        w, act = operands(gen(N), N, 300, 1040)
        want, _ = q6.f8_mmq(w, act, dtype=F32)
        codes = act.xq.view(torch.uint8)
        codes[1:] = 0x38
        Y, _ = q6.f8_mmq(w, act, dtype=F32)
        assert torch.equal(Y[0], want[0])


@pytest.mark.parametrize("N", [1, 12, 70, 500])
def test_repeated_calls_agree_bit_for_bit(N):
    w, act = operands(gen(N), N, 2056, 3600)
    want, _ = q6.f8_mmq(w, act, dtype=F32)
    for _ in range(20):
        Y, _ = q6.f8_mmq(w, act, dtype=F32)
        assert torch.equal(Y, want)


# ------------------------------------------------------------- in a program ---

class Block:
    """norm -> gate and up -> silu * up -> down -> norm with the residual, as a model's layers
    run them, in e4m3 blocks or (q8) K-quant weights."""

    def __init__(self, hidden, inner, seed=0):
        g = gen(seed)
        self.norm = (1 + 0.1 * randn(g, hidden)).bfloat16()
        self.up = (randn(g, 2 * inner, hidden) / hidden ** 0.5).bfloat16()
        self.down = (randn(g, hidden, inner) / inner ** 0.5).bfloat16()
        self.w_up, self.w_down = q6.f8_quantize_weights(self.up), q6.f8_quantize_weights(self.down)

    def __call__(self, y, h):
        """y: the output of the layers before, h: the residual stream (updated in place)."""
        act, h = q6.rms_norm_f8(y, self.norm, 1e-6, residual=h)
        gu, _ = q6.f8_mmq(self.w_up, act)
        y, _ = q6.f8_mmq(self.w_down, q6.silu_mul_f8(gu))
        return y, h

    def exact(self, y, h):
        h = h.double() + y.double()
        x = h * ((h * h).mean(1, keepdim=True) + 1e-6) ** -0.5 * self.norm.double()
        g, u = (x @ self.up.double().t()).chunk(2, dim=1)
        return (g * torch.sigmoid(g) * u) @ self.down.double().t(), h


@pytest.mark.parametrize("N", [1, 5, 33, 200])
def test_a_run_of_them_against_the_unquantised_steps(N):
    """Four quantisations, each off by up to 2^-4 of a value and about a third of that in the mean
    (uniform in a step whose length varies by 2: 2^-4 / sqrt(3) * 0.75 = 0.027 of the root mean
    square), two in each product: sqrt(2) * 0.027 = 0.038 in gate and up; their product's silu adds
    gate's and up's, sqrt(2) * 0.038 = 0.054 (silu's slope is within 1.1), the down product's two
    more: sqrt(0.054^2 + 0.038^2) = 0.07. Twice that is allowed for."""
    block = Block(1024, 1408)
    g = gen(N)
    y, h = randn(g, N, 1024).bfloat16(), randn(g, N, 1024).bfloat16()
    want, stream = block.exact(y, h)
    got, h2 = block(y, h)
    q6.sync_status()
    assert h2 is h
    assert ((h.double() - stream).abs() <= (2.0 ** -8 + 2 * ref.U) * stream.abs()).all()
    assert (got.double() - want).norm() <= 0.14 * want.norm()


@pytest.mark.parametrize("N", [1, 40])
def test_int8_activations_feed_the_k_quant_products(N):
    """What the norm and the gated activation make is what mmq() and q4k_mmq() take."""
    from q6_int8_mmq_gb300 import synth
    M, K = 256, 512
    w6 = q6.pack_weights(torch.from_numpy(synth.q6k_raw_weights(1, M, K)).cuda(), M, K)
    w4 = q6.q4k_pack_weights(torch.from_numpy(synth.q4k_raw_weights(2, M, K)).cuda(), M, K)
    g = gen(N)
    x, weight = randn(g, N, K), 1 + 0.1 * randn(g, K)
    act, _ = q6.rms_norm_q8(x, weight, 1e-6, want_us=True)
    y = x.double() * ((x.double() ** 2).mean(1, keepdim=True) + 1e-6) ** -0.5 * weight.double()
    plain = q6.quantize_act(y.float(), want_us=True)
    # the same values but for the last bits of the row's factor: a few codes may fall the other way
    for got, want in ((q6.mmq(w6, act)[0], q6.mmq(w6, plain)[0]),
                      (q6.q4k_mmq(w4, act)[0], q6.q4k_mmq(w4, plain)[0])):
        assert (got - want).norm() <= 1e-3 * want.norm()
    gu = torch.cat([x, x.flip(1)], 1)
    act = q6.silu_mul_q8(gu, want_us=True)
    plain = q6.quantize_act((torch.nn.functional.silu(x.double()) * x.flip(1).double()).float(),
                            want_us=True)
    assert (q6.mmq(w6, act)[0] - q6.mmq(w6, plain)[0]).norm() <= 1e-3 * q6.mmq(w6, plain)[0].norm()
    q6.sync_status()


@pytest.mark.parametrize("N", [1, 5, 40, 200])
def test_the_feed_forward_example(N):
    """Its layers against the unquantised steps: e4m3 as above; int8 codes of 32 values are off by up
    to 1/254 of the largest (3 of the root mean square), 0.3 of that in the mean: 0.004 for each of
    the two activations of a chain (gate and up add), 0.01 in all; four times that is allowed for."""
    from examples import feed_forward
    assert feed_forward.check(feed_forward.BlockLayer(512, 768), N, 512) <= 0.14
    assert feed_forward.check(feed_forward.KQuantLayer(512, 768), N, 512) <= 0.04


@pytest.mark.parametrize("N", [1, 33, 300])
def test_in_a_graph_and_on_another_stream(N):
    block = Block(512, 768)
    g = gen(N)
    y, h = randn(g, N, 512).bfloat16(), randn(g, N, 512).bfloat16()
    h0 = h.clone()
    want, _ = block(y, h)
    want_h = h.clone()
    side = torch.cuda.Stream()
    h.copy_(h0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = block(y, h)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(h, want_h)
    # an explicit stream argument, outputs allocated on it
    act, _ = q6.rms_norm_f8(y, block.norm, 1e-6, residual=h0.clone(), stream=side)
    out, _ = q6.f8_mmq(block.w_up, act, stream=side)
    side.synchronize()
    act2, _ = q6.rms_norm_f8(y, block.norm, 1e-6, residual=h0.clone())
    assert torch.equal(out, q6.f8_mmq(block.w_up, act2)[0])
    graphs = []
    for _ in range(2):
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out, _ = block(y, h)
        graphs.append((gr, out))
    for k in range(3):
        for gr, out in graphs:
            y.copy_(randn(g, N, 512))
            h.copy_(h0)
            gr.replay()
            h_got = h.clone()
            h.copy_(h0)
            eager, _ = block(y, h)
            assert torch.equal(out, eager) and torch.equal(h_got, h)
    q6.sync_status()


def test_back_to_back_products_of_changing_operands():
    """Kernels that start while the one before still runs read what it has written."""
    g = gen(8)
    acts = [activations(g, 40, 2048, BF16) for _ in range(8)]
    w = q6.f8_quantize_weights(randn(g, 1000, 2048))
    want = [q6.f8_mmq(w, q6.f8_quantize_act(x))[0].clone() for x in acts]
    buf, out = q6.alloc_f8_activations(40, 2048), torch.empty(40, 1000, dtype=BF16, device="cuda")
    wbuf = q6.alloc_f8_weights(1000, 2048)
    dense = randn(gen(9), 1000, 2048)
    wide = q6.f8_quantize_weights(dense)
    for k in range(40):
        q6.f8_quantize_act(acts[k % 8], out=buf)
        q6.f8_mmq(w, buf, out=out)
        assert torch.equal(out, want[k % 8])
        wbuf.wq.view(torch.uint8).zero_()
        q6.f8_quantize_weights(dense, out=wbuf)
        got, _ = q6.f8_mmq(wbuf, buf)
        assert torch.equal(got, q6.f8_mmq(wide, buf)[0])


@pytest.mark.parametrize("N,M", [(140, 1000), (140, 2056), (600, 1100)])
def test_shared_tiles_back_to_back_in_graphs_and_on_two_streams(N, M):
    """Products whose tiles several pairs of CTAs share, right behind what writes their operands."""
    K = 3600
    g = gen(M)
    xs = [activations(g, N, K, BF16) for _ in range(4)]
    w = q6.f8_quantize_weights(randn(g, M, K))
    want = [q6.f8_mmq(w, q6.f8_quantize_act(x))[0].clone() for x in xs]
    buf, out = q6.alloc_f8_activations(N, K), torch.empty(N, M, dtype=BF16, device="cuda")
    for k in range(24):
        q6.f8_quantize_act(xs[k % 4], out=buf)
        q6.f8_mmq(w, buf, out=out)
        got = out.clone()
        q6.f8_mmq(w, buf, out=out)
        assert torch.equal(got, want[k % 4]) and torch.equal(out, got)
    graphs = []
    for _ in range(2):
        x, torch_graph = xs[0].clone(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(torch_graph):
            act = q6.f8_quantize_act(x)
            ys = [q6.f8_mmq(w, act)[0] for _ in range(3)]
        graphs.append((torch_graph, x, ys, torch.cuda.Stream()))
    for k in range(6):
        for i, (gr, x, ys, stream) in enumerate(graphs):     # both at a time
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                x.copy_(xs[(k + i) % 4])
                gr.replay()
        for i, (gr, x, ys, stream) in enumerate(graphs):
            torch.cuda.current_stream().wait_stream(stream)
            assert all(torch.equal(y, want[(k + i) % 4]) for y in ys)
    q6.sync_status()


def test_offsets_past_32_bits():
    K, M, N = 16384, 270000, 3
    wq = torch.zeros(M, K, dtype=torch.uint8, device="cuda")       # 4.4 GB of codes
    sw = torch.ones(-(-M // 128), K // 128, device="cuda")
    g = gen(5)
    rows = [0, 1, 131071, 131072, 262143, 262144, 262145, M - 1]
    for r in rows:
        wq[r] = (0.5 * randn(g, K)).to(torch.float8_e4m3fn).view(torch.uint8)
    w = q6.F8Weights(M, K, wq.view(torch.float8_e4m3fn), sw)
    act = q6.f8_quantize_act(randn(g, N, K))
    Y, _ = q6.f8_mmq(w, act, dtype=F32)
    x = act.xq.double() * act.sx[:, :N].double().t().repeat_interleave(128, 1)
    part = w.wq.view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
    size = x.abs() @ part.abs().t()
    assert ((Y[:, rows].double() - x @ part.t()).abs() <= size * (132 + K / 128 + 3) * ref.U).all()
    Y[:, rows] = 0
    assert not Y.any()
    # rows of activations, and of the result, past 2^32 bytes
    N = M
    act = q6.F8Activations(N, K, w.wq, torch.ones(K // 128, N, device="cuda"))
    small = q6.f8_quantize_weights(randn(g, 24, K))
    Y, _ = q6.f8_mmq(small, act, dtype=BF16)
    want, bound = ref.product(w.wq.view(torch.uint8)[rows].view(torch.float8_e4m3fn),
                              torch.ones(K // 128, 8, device="cuda"), small.wq, small.sw, BF16)
    assert ((Y[rows].double() - want).abs() <= bound).all()
    Y[rows] = 0
    assert not Y.any()


def test_the_first_product_of_a_process_may_be_captured():
    """The kernels' limits of shared memory are raised by the first call that runs them, in a graph too."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, q6_int8_mmq_gb300 as q6
x = torch.ones(300, 512, device="cuda")
act, w = q6.f8_quantize_act(x), q6.f8_quantize_weights(x[:200])
out, few = torch.empty(300, 200, device="cuda"), torch.empty(3, 200, device="cuda")
small = q6.f8_quantize_act(x[:3])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q6.f8_mmq(w, act, out=out)
    q6.f8_mmq(w, small, out=few)
graph.replay()
torch.cuda.synchronize()
assert (out - 512).abs().max() < 1e-3 and (few - 512).abs().max() < 1e-3, (out, few)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, CUDA_MODULE_LOADING="LAZY"))
    assert r.returncode == 0, r.stdout + r.stderr


def test_calls_that_do_not_fit_are_refused():
    w, act = operands(gen(1), 3, 40, 512)
    x, weight = randn(gen(2), 3, 512), torch.ones(512, device="cuda")
    f8, q8 = q6.alloc_f8_activations(3, 256), q6.alloc_activations(2, 512)
    wide = torch.zeros(3, 1024, device="cuda")
    for call in (lambda: q6.f8_mmq(w, act, dtype=torch.float64),
                 lambda: q6.f8_mmq(w, act, out=torch.zeros(3, 41, device="cuda")),
                 lambda: q6.f8_mmq(w, act, out=torch.zeros(40, 3, device="cuda").t()),
                 lambda: q6.f8_mmq(w, act, out=torch.zeros(3, 40, dtype=torch.int32, device="cuda")),
                 lambda: q6.f8_mmq(w, act, out=torch.zeros(3, 40, device="cuda"), dtype=F16),
                 lambda: q6.f8_mmq(w, act, out=torch.zeros(3, 40)),                 # host memory
                 lambda: q6.f8_mmq(w, q6.f8_quantize_act(wide)),
                 lambda: q6.f8_quantize_act(x, out=f8),
                 lambda: q6.f8_quantize_act(x, out=q8),
                 lambda: q6.f8_quantize_weights(x, out=w),
                 lambda: q6.f8_quantize_act(x[:, :500]),
                 lambda: q6.f8_quantize_act(wide[:, 1:513]),                        # rows off 16 bytes
                 lambda: q6.silu_mul_q8(x, out=q8),                                 # K = 256, out has 512
                 lambda: q6.silu_mul_q8(wide, out=q8),
                 lambda: q6.silu_mul_f8(wide, out=f8),
                 lambda: q6.rms_norm_q8(x, weight, 1e-6, out=q8),
                 lambda: q6.rms_norm_q8(x, weight, 1e-6, want_xh=False, want_xq=False),
                 lambda: q6.rms_norm_f8(x, weight[:256], 1e-6),
                 lambda: q6.rms_norm_f8(x, weight.double(), 1e-6),
                 lambda: q6.rms_norm_f8(x, weight, 0.0),
                 lambda: q6.rms_norm_f8(x, weight, "small"),
                 lambda: q6.rms_norm_q8(x, weight, None),
                 lambda: q6.rms_norm_f8(x, weight, 1e-6, h=x),
                 lambda: q6.rms_norm_f8(x, weight, 1e-6, residual=x.half(), h=x),
                 lambda: q6.rms_norm_f8(x, weight, 1e-6, residual=wide),
                 lambda: q6.rms_norm_f8(x, weight, 1e-6, residual=x.cpu()),
                 lambda: q6.rms_norm_f8(x.t(), weight, 1e-6)):
        with pytest.raises(q6.Q6Error):
            call()


def test_another_device_than_the_current_one_is_refused():
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    x = torch.ones(2, 256, device="cuda:1")
    with pytest.raises(q6.Q6Error):
        q6.f8_quantize_act(x)
