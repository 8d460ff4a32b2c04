"""GPU tests of the codes that the norm, the gated activation and the quantisers end in: bit for bit
against their definition in f32, at ties, in the forms that prompts take, and past 2^32 bytes.

The definitions' f32 steps are one rounding each (sum, product, quotient, all IEEE), so the kernels have
nothing to choose: codes are compared for equality. The gated activation's exponential is the exception; its
codes are held to half of the step that lies at their value."""
import pytest

torch = pytest.importorskip("torch")

import q6_int8_mmq_gb300 as q6  # noqa: E402
import f8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
# every pair of the types of X and of the residual stream
PAIRS = [(t, r) for t in TYPES for r in (None, *TYPES)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def rows(g, N, K, dtype):
    """N(0, 1) with wide channels, rows of other sizes, an all-zero row and zero blocks."""
    x = randn(g, N, K) * torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 20.0, 1.0)
    x = x * torch.exp(randn(g, N, 1))
    if N > 2:
        x[1] = 0
        x[2, :min(K, 160)] = 0
    return x.to(dtype)


def over(a, b):
    """a / b in f32; a or b may be a number (as a tensor, so that it is a division)."""
    full = a if isinstance(a, torch.Tensor) else b
    a, b = (v if isinstance(v, torch.Tensor) else torch.full_like(full, v) for v in (a, b))
    return a / b


E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()     # 0 to 448


def e4m3_of(u):
    """The nearest e4m3 values of f32 values of at most 448 or a rounding more, ties to the even code."""
    table = E4M3.to(u.device)
    middle = (table[:-1] + table[1:]) / 2
    a = u.abs().double()
    at = torch.searchsorted(middle, a)                     # middle[at - 1] < a <= middle[at]
    tie = (at < 126) & (a == middle[at.clamp(max=125)]) & (at % 2 == 1)
    return table[at + tie.long()] * torch.sign(u)


def f8_of(t, side=1):
    """f32 t [N, K] -> the e4m3 values of its codes (f64) and scales [N / side, K / 128] (f32)."""
    N, K = t.shape
    top, each = ref.block_max(t, side, 128)
    live = top >= 2.0 ** -100
    by = torch.where(live, over(448.0, top), 0.0)
    by = by.repeat_interleave(side, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return e4m3_of(t * by), torch.where(live, over(top, 448.0), 0.0)


def q8_of(t):
    """f32 t [N, K] -> int8 codes (f64) and scales [N, K / 32] (f32)."""
    b = t.unflatten(1, (-1, 32))
    d = over(b.abs().amax(2), 127.0)
    q = torch.where(d.unsqueeze(2) > 0, b / d.unsqueeze(2), 0.0).double()
    return (torch.sign(q) * (q.abs() + 0.5).floor().clamp(max=127)).flatten(1), d


def f8_codes(act):
    return act.xq.double()


def check_f8(act, N, t, factor=None, factor_rel=0.0):
    """Codes bit for bit; scales too, or (factor: the rows' 1 / rms in f64, within factor_rel) within
    the factor's error, its rounding to f32 and the product's."""
    codes, d = f8_of(t)
    assert torch.equal(f8_codes(act), codes)
    check_scales(act.sx[:, :N].t(), d, factor, factor_rel)


def check_q8(act, N, t, factor=None, factor_rel=0.0):
    codes, d = q8_of(t)
    for got in (act.xq, act.xh):
        assert got is None or torch.equal(got.double(), codes)
    check_scales(act.da[:, :N].t(), d, factor, factor_rel)
    if act.us is not None:
        pairs = act.us.double()
        got = pairs.unflatten(1, (-1, 2, 8))[:, :act.K // 256].sum(2).flatten(1)
        want = act.da[:, :N].t().double() * codes.unflatten(1, (-1, 32)).sum(2)
        assert ((got - want).abs() <= ref.U * want.abs()).all()


def check_scales(got, d, factor, factor_rel):
    if factor is None:
        assert torch.equal(got, d)
    else:
        want = d.double() * factor
        assert ((got.double() - want).abs() <= want * (factor_rel + 2 * ref.U)).all()


# ------------------------------------------------------------------- ties ---

def e4m3_ties(dtype):
    """Rows of 128 whose largest value is 448, so that their codes are those of the values: every value
    halfway between two codes, of both signs, and the values next to it."""
    table = E4M3.cuda()
    middle = (table[:-1] + table[1:]) / 2
    if dtype is F32:
        step = middle * 2.0 ** -18
        middle = torch.cat([middle, middle + step, middle - step])
    values = torch.cat([middle, -middle])
    values = torch.nn.functional.pad(values, (0, -values.numel() % 127)).view(-1, 127)
    x = torch.cat([values, torch.full_like(values[:, :1], 448.0)], 1).to(dtype)
    assert torch.equal(x[:, :127].double(), values)
    return x


def int8_ties(dtype):
    """Rows of 256, blocks of 32 whose largest value is 127: every half, of both signs."""
    half = torch.arange(127, device="cuda").double() + 0.5
    if dtype is F32:
        half = torch.cat([half, half * (1 + 2.0 ** -20), half * (1 - 2.0 ** -20)])
    values = torch.cat([half, -half])
    values = torch.nn.functional.pad(values, (0, -values.numel() % 31)).view(-1, 31)
    blocks = torch.cat([values, torch.full_like(values[:, :1], 127.0)], 1)
    blocks = torch.cat([blocks, blocks[:1].expand(-blocks.shape[0] % 8, 32)])
    x = blocks.reshape(-1, 256).to(dtype).float()
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_e4m3_ties_go_to_the_even_code(dtype):
    x = e4m3_ties(dtype)
    N = x.shape[0]
    ones = torch.ones(128, device="cuda")
    table = E4M3.cuda()
    codes = q6.f8_quantize_act(x).xq.view(torch.uint8)
    half = (x[:, :127].abs().double().unsqueeze(2) == (table[:-1] + table[1:]) / 2).any(2)
    assert half.sum() >= 252 and not (codes[:, :127][half] & 1).any()
    for act in (q6.f8_quantize_act(x), q6.rms_norm_f8(x, ones, 1e-6)[0],
                q6.rms_norm_f8(torch.zeros_like(x), ones, 1e-6, residual=x.float())[0]):
        assert torch.equal(act.xq.view(torch.uint8), codes)
    check_f8(q6.f8_quantize_act(x), N, x.float())
    assert (q6.f8_quantize_act(x).sx[:, :N] == 1).all()
    w = q6.f8_quantize_weights(x)
    assert torch.equal(w.wq.view(torch.uint8), codes) and (w.sw == 1).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_int8_ties_go_away_from_zero(dtype):
    x = int8_ties(dtype)
    act, _ = q6.rms_norm_q8(x, torch.ones(256, device="cuda"), 1e-6)
    u = x.double()
    tie = (u.abs() % 1) == 0.5
    assert tie.sum() >= 254
    assert torch.equal(act.xq.double()[tie], (torch.sign(u) * (u.abs() + 0.5))[tie])
    root = ((u * u).mean(1, keepdim=True) + 1e-6) ** -0.5
    check_q8(act, x.shape[0], x.float(), root, ref.norm(x, None, torch.ones(256, device="cuda"), 1e-6)[4])


# ------------------------------------------- codes, in the forms of prompts ---

def check_norm(N, K, type, rtype, f8):
    g = gen(N + K)
    x = rows(g, N, K, type)
    r = None if rtype is None else (2 * rows(g, N, K, F32)).to(rtype)
    w = (1 + 0.3 * randn(g, K)).to(TYPES[(N + TYPES.index(type)) % 3])
    _, _, root, _, root_rel = ref.norm(x, r, w, 1e-5)
    h32 = x.float() if r is None else x.float() + r.float()
    want_h = None if r is None else h32.to(rtype)
    if f8:
        act, h = q6.rms_norm_f8(x, w, 1e-5, residual=r)
        check_f8(act, N, h32 * w.float(), root, root_rel)
    else:
        act, h = q6.rms_norm_q8(x, w, 1e-5, residual=r, want_us=True)
        check_q8(act, N, h32 * w.float(), root, root_rel)
    assert h is (x if r is None else r) and (r is None or torch.equal(h, want_h))


@pytest.mark.parametrize("type,rtype", PAIRS)
def test_norm_codes_in_every_form(type, rtype):
    """A part of a row a warp: few rows, many; and two parts a warp, from 2^23 values on, the second past
    the row's end in some warps and cut by it in one."""
    for f8, sizes in ((True, ((3, 400), (200, 1040), (2050, 4112), (1100, 7696))),
                      (False, ((3, 512), (200, 1280), (2000, 4352), (1100, 7680)))):
        for N, K in sizes:
            check_norm(N, K, type, rtype, f8)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("N,K", [(3, 400), (2500, 1040), (640, 4656), (300, 8704), (5000, 528)])
def test_quantiser_codes_in_every_form(N, K, type):
    """One part of a row a warp, and (1.25 million f32 values, 2.5 million of 16 bits on) up to four,
    some of them past the row's end or cut by it."""
    x = rows(gen(N), N, K, type)
    big = torch.full((N, K + 8), float("nan"), dtype=type, device="cuda")
    big[:, :K] = x
    check_f8(q6.f8_quantize_act(x), N, x.float())
    check_f8(q6.f8_quantize_act(big[:, :K]), N, x.float())


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (300, 1040), (3000, 2064)])
def test_weight_codes(M, K, type):
    W = rows(gen(M), M, K, type)
    codes, d = f8_of(W.float(), 128)
    w = q6.f8_quantize_weights(W)
    assert torch.equal(w.wq.double(), codes) and torch.equal(w.sw, d)


def check_near(codes, scale, t, rel, f8):
    """Codes of values that the kernel knows within rel: off by at most half of the step at their value,
    and what rel, the largest value's rel and three roundings make of it."""
    top, each = ref.block_max(t, 1, 128 if f8 else 32)
    _, top_rel = ref.block_max(torch.where(t.abs() >= 0.99 * each, rel, 0.0), 1, 128 if f8 else 32)
    d = each / (448.0 if f8 else 127.0)
    u = torch.where(each >= (2.0 ** -100 if f8 else 2.0 ** -140), t / d, 0.0)
    half = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 4) if f8 else 0.5
    slack = u.abs() * (rel + top_rel + 4 * ref.U)
    assert ((codes - u).abs() <= half + slack).all(), float(((codes - u).abs() - half - slack).max())
    want = top / (448.0 if f8 else 127.0)
    bound = want * (top_rel[:, ::128 if f8 else 32] + 2 * ref.U)
    assert ((scale - want).abs() <= bound).all()


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("f8,N,K", [(True, 3, 400), (True, 1300, 1040), (True, 330, 4656), (False, 3, 512),
                                    (False, 1100, 1280), (False, 330, 4864)])
def test_activation_codes_in_every_form(f8, N, K, type):
    """One part of a row a warp, and (0.6 million int8 codes of f32 rows, 1.2 million codes of 16-bit rows
    on) two, the second past the row's end or cut by it."""
    x = rows(gen(N), N, 2 * K, type)
    t, rel = ref.silu_mul(x)
    if f8:
        act = q6.silu_mul_f8(x)
        check_near(f8_codes(act), act.sx[:, :N].t().double(), t, rel, True)
    else:
        act = q6.silu_mul_q8(x, want_us=True)
        check_near(act.xh.double(), act.da[:, :N].t().double(), t, rel, False)
        assert torch.equal(act.xh, act.xq.half())
        again = q6.silu_mul_q8(x, want_xh=False)
        assert torch.equal(again.xq, act.xq) and torch.equal(again.da[:, :N], act.da[:, :N])


def test_gates_far_below_zero():
    """silu(g) is within 2^-16 of its value at g = -87 and 0 below -87.34, where 1 + exp(-g) is above
    2^126."""
    g = torch.tensor([-87.0, -87.3, -87.4, -88.0, -89.0, -150.0, -3e38], device="cuda")
    x = torch.cat([g[:, None].expand(-1, 256), torch.full((7, 256), 1e30, device="cuda")], 1)
    act = q6.silu_mul_q8(x)
    y = act.xq.double() * act.da[:, :7].t().double().repeat_interleave(32, 1)
    want = (g[:2].double() * torch.sigmoid(g[:2].double()) * torch.tensor(1e30).double().item())[:, None]
    assert ((y[:2] - want).abs() <= 2.0 ** -16 * want.abs()).all()
    assert not act.xq[2:].any() and not act.da[:, 2:7].any()


# ------------------------------------------------------- past 2^32 bytes ---

def test_rows_of_codes_past_32_bits():
    """More than 2^32 codes: rows on both sides of that are what a call of those rows alone makes."""
    K = 16640
    N = 2 ** 32 // K + 500
    at = [0, 1, N // 2, 2 ** 32 // K - 1, 2 ** 32 // K, 2 ** 32 // K + 1, N - 1]
    some = rows(gen(1), len(at), 2 * K, BF16)
    some[some == 0] = 1                                    # no zeros, so that no row is left out
    weight = 1 + 0.1 * randn(gen(2), K)

    def check(act, want, exact=True):
        codes = act.xq if act.xq is not None else act.xh
        scale, want_scale = (act.sx, want.sx) if hasattr(act, "sx") else (act.da, want.da)
        few = want.xq if act.xq is not None else want.xh
        assert torch.equal(codes[at].float(), few.float())
        got, small = scale[:, at], want_scale[:, :len(at)]
        if exact:
            assert torch.equal(got, small)
        else:      # the row's sum of squares is added in another order: each side's bound
            bound = 2 * (((K / 256 + 48) / 2 + 4) * ref.U + 2 * ref.U)
            assert ((got - small).abs() <= bound * small).all()
        codes[at] = 0
        scale[:, at] = 0
        assert not codes.view(torch.uint8 if codes.element_size() == 1 else torch.int16).any()
        assert not scale[:, :N].any()

    x = torch.zeros(N, 2 * K, dtype=BF16, device="cuda")   # 17 GB
    x[at] = some
    check(q6.silu_mul_f8(x), q6.silu_mul_f8(some))
    check(q6.silu_mul_q8(x, want_xq=False), q6.silu_mul_q8(some))
    x = x.view(2 * N, K)[:N]
    x.zero_()
    some = some[:, :K].contiguous()
    x[at] = some
    check(q6.f8_quantize_act(x), q6.f8_quantize_act(some))
    r = torch.zeros(N, K, dtype=BF16, device="cuda")
    act, h = q6.rms_norm_f8(x, weight, 1e-6, residual=r)
    assert h is r and torch.equal(h[at], some)
    check(act, q6.rms_norm_f8(some, weight, 1e-6)[0], exact=False)
    h[at] = 0
    assert not h.view(torch.int16).any()
    w = q6.f8_quantize_weights(x)
    codes, d = f8_of(x[-(N % 128 or 128):].float(), 128)
    assert torch.equal(w.wq[-(N % 128 or 128):].double(), codes) and torch.equal(w.sw[-1:], d)
    assert w.wq.view(torch.uint8)[at].any(1).all()
    w.wq[at] = 0
    assert not w.wq.view(torch.uint8).any()


@pytest.mark.parametrize("N,M,K,dtype,ld", [(70, 40, 272, BF16, 2 ** 25), (70, 300, 272, F32, 2 ** 24),
                                            (70, 40, 272, F16, 2 ** 25 + 1), (70, 300, 272, BF16, 2 ** 25 + 2),
                                            (70, 40, 272, F32, 2 ** 24 + 1), (70, 40, 3600, BF16, 2 ** 25),
                                            (64, 40, 1040, BF16, 2 ** 25 + 2 ** 22), (64, 40, 112, F32, 2 ** 24 + 2 ** 21)])
def test_results_past_32_bits(N, M, K, dtype, ld):
    """Rows of Y far apart: its last ones lie past 2^32 bytes, stored by TMA and in words of 4 and 2 bytes,
    with shared tiles and by the few-token kernel; nothing is written between them."""
    g = gen(N + M)
    w = q6.f8_quantize_weights(randn(g, M, K))
    act = q6.f8_quantize_act(randn(g, N, K))
    want, _ = q6.f8_mmq(w, act, dtype=dtype)
    big = torch.zeros(N * ld, dtype=dtype, device="cuda")
    Y = torch.as_strided(big, (N, M), (ld, 1))
    assert (N - 1) * ld * big.element_size() > 2 ** 32
    got, _ = q6.f8_mmq(w, act, out=Y)
    q6.sync_status()
    assert got is Y and torch.equal(Y, want)
    Y.zero_()
    assert not big.view(torch.int16 if big.element_size() == 2 else torch.int32).any()
