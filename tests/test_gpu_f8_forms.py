"""Which kernel takes a product of e4m3 blocks: each of them runs at the sizes meant for it, and is right
there."""
import pytest

torch = pytest.importorskip("torch")

import q6_int8_mmq_gb300 as q6  # noqa: E402
import f8_reference as ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_sizes_are_refused_as_by_the_product():
    for M, K, N in ((0, 512, 3), (64, 40, 3), (64, 0, 3), (64, 512, -1), (2 ** 31 - 1, 16, 1),
                    (2 ** 30, 16, 2 ** 30), (2 ** 32 + 64, 512, 3), (64, 512, 2 ** 32 + 3)):
        with pytest.raises(q6.Q6Error):
            q6.f8_mmq_form(M, K, N)
    assert q6.f8_mmq_form(64, 512, 0) == ("none", 0, 0, 0, 0)
    assert q6.load().q6_f8_mmq_form(64, 512, 0, None, None, None, None, None) == q6.Q6_EINVAL


# (N, M, K) -> path, tokens and rows of a tile, parts of K
FORMS = [((1, 128, 128), ("f8_few", 16, 128, 1)),        # a single block of K
         ((16, 300, 400), ("f8_few", 16, 128, 4)),       # as many parts as blocks
         ((17, 1000, 2064), ("f8_few", 32, 128, 8)),
         ((32, 2056, 1040), ("f8_few", 32, 128, 8)),
         ((33, 8000, 1040), ("f8_few", 64, 128, 4)),
         ((64, 22016, 528), ("f8_few", 64, 128, 1)),     # more bands than the SMs take in two parts
         ((65, 1024, 1152), ("f8_tc", 256, 128, 1)),     # few tiles, a short K
         ((65, 1024, 3600), ("f8_tc", 256, 128, 4)),
         ((300, 1300, 3600), ("f8_tc", 256, 128, 2)),
         ((2048, 4096, 528), ("f8_tc", 256, 256, 1))]


def check_exact(N, M, K):
    """Codes -4 .. 4 and scales that are powers of two: every sum fits f32, so the result is exact."""
    g = torch.Generator(device="cuda").manual_seed(N)
    small = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    power = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g, device="cuda").float())  # noqa: E731
    act = q6.F8Activations(N, K, small(N, K).to(torch.float8_e4m3fn), power(-(-K // 128), -(-N // 4) * 4))
    w = q6.F8Weights(M, K, small(M, K).to(torch.float8_e4m3fn), power(-(-M // 128), -(-K // 128)))
    Y, path = q6.f8_mmq(w, act, dtype=torch.float32)
    q6.sync_status()
    assert torch.equal(Y.double(), ref.product(act.xq, act.sx, w.wq, w.sw, torch.float32)[0])
    return path


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,form", FORMS)
def test_every_form_runs_where_it_is_meant_to(sizes, form):
    N, M, K = sizes
    chosen = q6.f8_mmq_form(M, K, N)
    assert chosen[:4] == form and chosen.room > 0
    assert check_exact(N, M, K) == form[0]


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 17, 64])
@pytest.mark.parametrize("K", [384, 1024, 4096])
def test_all_clusters_of_a_few_tokens_run_at_a_time(N, K):
    """A cluster that has to wait for others to end reads its weights alone: 37 bands of weights in
    eight parts each took 9.1 us where 36 took 6.4."""
    for bands in range(1, 320):
        form = q6.f8_mmq_form(128 * bands, K, N)
        assert form.path == "f8_few" and 1 <= form.parts <= 8
        assert form.parts == 1 or bands <= form.room, (bands, form)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 17, 64])
@pytest.mark.parametrize("parts", range(1, 9))
def test_every_number_of_parts_is_exact(N, parts):
    """The largest weight that is split into this many parts, and a row less."""
    K = 1040
    bands = [b for b in range(1, 320) if q6.f8_mmq_form(128 * b, K, N).parts == parts]
    if not bands:
        pytest.skip("this device has as much room for clusters of one more")
    for M in (128 * bands[-1], 128 * bands[-1] - 127):
        assert q6.f8_mmq_form(M, K, N).parts == parts
        check_exact(N, M, K)


@pytest.mark.gpu
@pytest.mark.parametrize("N,M,K", [(5, 300, 1040), (40, 1000, 528), (70, 300, 528), (70, 1024, 3600),
                                   (300, 1000, 3600), (2048, 4096, 400)])
def test_infinite_and_nan_scales_go_through_the_formula(N, M, K):
    """What 64-bit arithmetic makes of the blocks' sums, infinities and NaN of them in the same places."""
    g = torch.Generator(device="cuda").manual_seed(M)
    blocks, inf, nan = -(-K // 128), float("inf"), float("nan")
    x = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (M, K), generator=g, device="cuda").float()
    x[3, 128:256] = 0                                     # a block whose sum is 0
    sx, sw = torch.ones(blocks, -(-N // 4) * 4, device="cuda"), torch.ones(-(-M // 128), blocks, device="cuda")
    sx[0, 0] = inf                                        # meets sums of both signs, and zeros
    sx[1, 1], sx[2, 1], sx[1, 3] = -inf, 0.0, inf
    sx[0, 4] = nan
    sw[0, 1] = inf                                        # the first 128 rows
    if M > 128:
        sw[-1, 2] = nan
    act = q6.F8Activations(N, K, x.to(torch.float8_e4m3fn), sx)
    weight = q6.F8Weights(M, K, w.to(torch.float8_e4m3fn), sw)
    Y, _ = q6.f8_mmq(weight, act, dtype=torch.float32)
    q6.sync_status()
    want = torch.zeros(N, M, dtype=torch.float64, device="cuda")
    for b in range(blocks):
        at = slice(128 * b, min(128 * b + 128, K))
        each = sx[b, :N].double()[:, None] * sw[:, b].double().repeat_interleave(128)[:M]
        want += each * (x[:, at].double() @ w[:, at].double().t())
    assert torch.equal(Y.isnan(), want.isnan())
    assert torch.equal(Y.double().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    assert want.isnan().any() and (want == inf).any() and (want == -inf).any() and want[2].isfinite().any()
