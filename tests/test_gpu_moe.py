"""Expert routing, grouping, grouped K-quant products, combination and low-rank adapters against
64-bit references (GPU)."""
import numpy as np
import pytest

import q6_int8_mmq_gb300 as q6
from q6_int8_mmq_gb300 import synth

import moe_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def rng(request):
    return np.random.default_rng(list(request.node.name.encode()))


def cuda(a, type=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if type is None else t.to(TYPE[type])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    off = np.abs(got - want) > bound
    assert not off.any(), (f"{off.sum()} of {off.size} values off, first at {np.argwhere(off)[0]}: "
                           f"{got[off][0]} for {want[off][0]}, bound {bound[off][0]}")


def raw_experts(seed, fmt, E, M, K):
    make = synth.q4k_raw_weights if fmt == "q4_K" else synth.q6k_raw_weights
    return np.stack([make(seed + e, M, K) for e in range(E)])


# ------------------------------------------------------------------- route ---

def logits_with_cases(rng, N, E):
    x = rng.standard_normal((N, E)).astype(np.float32)
    x = np.round(x * 4) / 4                                   # many ties, and +0 and -0
    x[rng.random((N, E)) < 0.2] = -np.inf
    if N > 4:
        x[1] = -np.inf                                        # nothing left
        x[2] = np.finfo(np.float32).min                       # the lowest value is a choice
        x[3, rng.integers(E)] = np.nan
        x[4, 0] = np.inf
    return x


@pytest.mark.parametrize("N,E,topk", [(1, 64, 8), (1, 1, 1), (7, 3, 3), (33, 31, 4), (64, 8, 8),
                                      (65, 256, 8), (300, 100, 5), (1000, 1024, 32), (2049, 128, 6)])
@pytest.mark.parametrize("type,renorm", [("f32", True), ("bf16", False), ("f16", True)])
def test_route(rng, N, E, topk, type, renorm):
    x = cuda(logits_with_cases(rng, N, E), type)
    r = q6.moe_route(x, topk, renormalize=renorm)
    ids, weights = ref.route(f64(x), topk, renorm)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = f64(r.weights)
    assert np.array_equal(np.isnan(got), np.isnan(weights))
    # f32: an exponential (2 ulp), a sum of E terms, a division
    fine = ~np.isnan(weights)
    assert np.all(np.abs(got - weights)[fine] <= weights[fine] * (8 + E / 32) * 2.0 ** -23)
    offsets, rows, pos = ref.group(ids, E)
    assert np.array_equal(r.groups.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.groups.rows.cpu().numpy(), rows)
    assert np.array_equal(r.groups.pos.cpu().numpy(), pos)


def test_route_of_no_tokens():
    r = q6.moe_route(torch.empty((0, 5), device="cuda"), 2)
    assert r.groups.offsets.tolist() == [0] * 7


def test_route_reads_rows_of_a_wider_tensor(rng):
    wide = cuda(rng.standard_normal((40, 50)), "f32")
    r = q6.moe_route(wide[:, 3:23], 4)
    ids, _ = ref.route(f64(wide[:, 3:23]), 4, True)
    assert np.array_equal(r.ids.cpu().numpy(), ids)


@pytest.mark.parametrize("N,per_row,groups", [(1, 1, 1), (0, 2, 4), (500, 1, 7), (513, 1, 1024),
                                              (129, 4, 33), (5000, 3, 5)])
def test_group_rows(rng, N, per_row, groups):
    ids = rng.integers(-2, groups + 2, (N, per_row)).astype(np.int32)
    if N == 5000:
        ids[:] = 3                                            # all in one group
    g = q6.group_rows(cuda(ids), groups)
    offsets, rows, pos = ref.group(ids, groups)
    assert np.array_equal(g.offsets.cpu().numpy(), offsets)
    assert np.array_equal(g.rows.cpu().numpy(), rows)
    assert np.array_equal(g.pos.cpu().numpy(), pos)


# ----------------------------------------------------------------- experts ---

def run_experts(rng, fmt, type, ids, E, M, K, swiglu, gather, seed=5, pad=0):
    raw = raw_experts(seed, fmt, E, M, K)
    rows = ids.shape[0] if gather else ids.size
    X = cuda(rng.standard_normal((rows, K + pad)), type)[:, :K]
    w = q6.pack_experts(cuda(raw), fmt, E, M, K, swiglu=swiglu)
    g = q6.group_rows(cuda(ids.astype(np.int32)), E)
    Y, path = q6.experts_mmq(w, X, g, gather=gather)
    q6.sync_status()
    want, bound = ref.experts(raw, fmt, f64(X), ids, E, swiglu, gather, type)
    check(Y, want, bound)
    # random roundings: the whole result is far closer than the bound of each value
    size = np.linalg.norm(want)
    assert np.linalg.norm(f64(Y) - want) <= 4 * ref.ROUND[type] * size
    return path


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("N,topk,E,M,K,swiglu,gather", [
    (1, 1, 1, 1, 256, False, True), (1, 2, 4, 34, 512, True, True), (5, 3, 3, 129, 768, False, False),
    (40, 2, 6, 130, 1024, True, True), (17, 4, 7, 200, 2560, False, True),
    (150, 2, 3, 258, 512, True, False), (300, 1, 2, 127, 256, False, True),
])
def test_experts(rng, fmt, type, N, topk, E, M, K, swiglu, gather):
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(N)])
    run_experts(rng, fmt, type, ids, E, M, K, swiglu, gather)


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("counts", [[8], [9, 0, 16], [0, 0, 33, 1], [15, 17, 31, 32], [257, 0, 1],
                                    [64, 65, 255, 256]])
def test_experts_group_sizes(rng, fmt, counts):
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)])
    run_experts(rng, fmt, "bf16", rng.permutation(ids)[:, None], len(counts), 144, 512, False, True)


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,swiglu,gather", [(130, 512, True, True), (129, 768, False, False)])
def test_experts_few_but_crowded(rng, fmt, type, M, K, swiglu, gather):
    """No more items than experts, but in a few of them: 1, 7, 8, 9, 17 and none."""
    E = 45
    counts = np.zeros(E, int)
    counts[[0, 3, 4, 20, 44]] = 1, 9, 7, 17, 8
    ids = np.concatenate([np.repeat(np.arange(E), counts), np.full(3, -1)])
    path = run_experts(rng, fmt, type, rng.permutation(ids)[:, None], E, M, K, swiglu, gather)
    assert path == "experts_few"


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
def test_experts_few_nonfinite_token_stays_alone(rng, fmt):
    raw = raw_experts(4, fmt, 16, 40, 512)
    w = q6.pack_experts(cuda(raw), fmt, 16, 40, 512)
    g = q6.group_rows(cuda(np.full((12, 1), 9, np.int32)), 16)
    X = cuda(rng.standard_normal((12, 512)), "bf16")
    good = q6.experts_mmq(w, X, g)[0].clone()
    X[1, 7], X[10, 300] = float("inf"), float("nan")
    Y, path = q6.experts_mmq(w, X, g)
    assert path == "experts_few"
    assert not torch.isfinite(Y[1]).any() and torch.isnan(Y[10]).all()
    rest = [n for n in range(12) if n not in (1, 10)]
    assert torch.equal(Y[rest], good[rest])


@pytest.mark.parametrize("E", [256, 257, 1024])
@pytest.mark.parametrize("type", ["bf16", "f16"])
def test_experts_many_uneven(rng, E, type):
    """Tiles of every size over as many experts as there may be."""
    counts = np.ones(E, int)
    counts[[3, 4, E // 2, E - 1]] = 140, 300, 0, 190
    ids = rng.permutation(np.repeat(np.arange(E), counts))
    path = run_experts(rng, "q4_K", type, ids[:, None], E, 40, 256, False, True)
    assert path == "experts_tc"


@pytest.mark.parametrize("fmt,K", [("q4_K", 18944), ("q6_K", 11008)])
def test_experts_long_k(rng, fmt, K):
    run_experts(rng, fmt, "bf16", rng.integers(0, 2, (21, 1)), 2, 48, K, False, True)


@pytest.mark.parametrize("N", [6, 400])
def test_experts_without_an_expert(rng, N):
    """Items of no expert get zeros, rows behind them included."""
    ids = rng.integers(-1, 3, (N, 2))
    ids[-1] = -1
    run_experts(rng, "q6_K", "bf16", ids, 3, 72, 512, False, True)


@pytest.mark.parametrize("N", [3, 600])
def test_experts_strided_rows(rng, N):
    run_experts(rng, "q4_K", "bf16", rng.integers(0, 4, (N, 1)), 4, 64, 512, True, True, pad=24)


@pytest.mark.parametrize("N", [4, 500])
@pytest.mark.parametrize("fmt,type", [("q4_K", "bf16"), ("q6_K", "f16")])
def test_experts_wide_range(rng, N, fmt, type):
    """Tokens and rows whose sizes lie far apart keep their own precision."""
    E, M, K = 2, 96, 512
    raw = raw_experts(9, fmt, E, M, K)
    at = 0 if fmt == "q4_K" else 208
    blocks = raw.reshape(E, M, -1, ref.BLOCK[fmt])
    d = np.array([2.0 ** (e % 20 - 18) for e in range(M)], np.float16)   # row by row
    blocks[..., at:at + 2] = d.view(np.uint8).reshape(M, 1, 2)
    if fmt == "q4_K":
        blocks[..., 2:4] = (d / 2).view(np.uint8).reshape(M, 1, 2)
    ids = rng.integers(0, E, (N, 1))
    sizes = 2.0 ** (rng.integers(-40, 40, (N, 1)) if type == "bf16" else rng.integers(-4, 3, (N, 1)))
    X = cuda(rng.standard_normal((N, K)) * sizes, type)
    w = q6.pack_experts(cuda(raw), fmt, E, M, K)
    Y, _ = q6.experts_mmq(w, X, q6.group_rows(cuda(ids.astype(np.int32)), E))
    want, bound = ref.experts(raw, fmt, f64(X), ids, E, False, True, type)
    keep = np.abs(want) < 60000 if type == "f16" else np.full(want.shape, True)
    check(torch.where(cuda(keep), Y.double(), 0.0), np.where(keep, want, 0), bound)


@pytest.mark.parametrize("fmt", ["q4_K", "q6_K"])
@pytest.mark.parametrize("type,first,step", [("bf16", 0, 3), ("bf16", 0, 1), ("f16", -8, 1)])
@pytest.mark.parametrize("N,E", [(96, 2), (16, 24)])
def test_experts_super_blocks_far_apart(rng, fmt, type, first, step, N, E):
    """A row's super-blocks may differ by 2^21 in size, and a token may look at the small ones
    alone. Bound, beside a result's rounding: a weight's two terms and their sum are each rounded to
    11 bits, and the weight is off by 2^-12 of its super-block's largest possible weight."""
    M, K = 72, 2048
    raw = raw_experts(11, fmt, E, M, K)
    blocks = raw.reshape(E, M, K // 256, ref.BLOCK[fmt])
    d = np.array([2.0 ** (first - step * s) for s in range(K // 256)], np.float16)
    at = 0 if fmt == "q4_K" else 208
    blocks[..., at:at + 2] = d.view(np.uint8).reshape(-1, 2)
    if fmt == "q4_K":
        blocks[..., 2:4] = (-d).view(np.uint8).reshape(-1, 2)
    largest = np.abs(d.astype(np.float64)) * (945 + 63 if fmt == "q4_K" else 4096)
    x = np.zeros((N, K))
    mine = np.arange(N) % (K // 256)                    # the super-block a token looks at
    for n in range(N):
        x[n, 256 * mine[n]:256 * mine[n] + 256] = rng.standard_normal(256)
    ids = rng.integers(0, E, (N, 1))
    X = cuda(x, type)
    w = q6.pack_experts(cuda(raw), fmt, E, M, K)
    g = q6.group_rows(cuda(ids.astype(np.int32)), E)
    Y, path = q6.experts_mmq(w, X, g)
    assert path == ("experts_tc" if N > E else "experts_few")
    want, _ = ref.experts(raw, fmt, f64(X), ids, E, False, True, type)
    rows = g.rows.cpu().numpy()
    size = np.abs(f64(X)).sum(1) * largest[mine]
    bound = ref.ROUND[type] * np.abs(want) + ((3 * 2.0 ** -11 + 2.0 ** -12) * size)[rows][:, None]
    check(Y, want, bound)
    for s in range(K // 256):                           # and as a whole, as in run_experts
        of = mine[rows] == s
        off = np.linalg.norm((f64(Y) - want)[of])
        assert off <= 4 * ref.ROUND[type] * np.linalg.norm(want[of])


def test_experts_nonfinite_token_stays_alone(rng):
    """A token with an infinity or a NaN leaves the others as they are."""
    raw = raw_experts(4, "q4_K", 2, 40, 512)
    w = q6.pack_experts(cuda(raw), "q4_K", 2, 40, 512)
    for N in (4, 300):
        g = q6.group_rows(cuda(np.zeros((N, 1), np.int32)), 2)
        X = cuda(rng.standard_normal((N, 512)), "bf16")
        good = q6.experts_mmq(w, X, g)[0].clone()
        X[1, 7], X[2, 300] = float("inf"), float("nan")
        Y, _ = q6.experts_mmq(w, X, g)
        assert not torch.isfinite(Y[1]).any() and torch.isnan(Y[2]).all()
        rest = [n for n in range(N) if n not in (1, 2)]
        assert torch.equal(Y[rest], good[rest])


def test_experts_many_groups(rng):
    run_experts(rng, "q4_K", "bf16", rng.integers(0, 700, (50, 2)), 700, 16, 256, False, True)


def test_experts_repeats(rng):
    """The same call gives the same bits."""
    w = q6.pack_experts(cuda(raw_experts(3, "q6_K", 4, 300, 1024)), "q6_K", 4, 300, 1024)
    for N in (9, 700):
        X = cuda(rng.standard_normal((N, 1024)), "bf16")
        g = q6.group_rows(cuda(rng.integers(0, 4, (N, 1)).astype(np.int32)), 4)
        a = q6.experts_mmq(w, X, g)[0]
        for _ in range(3):
            assert torch.equal(a, q6.experts_mmq(w, X, g)[0])


# ------------------------------------------------------------------ combine ---

@pytest.mark.parametrize("N,topk,M", [(1, 1, 1), (3, 8, 64), (33, 2, 2056), (100, 5, 999),
                                      (257, 32, 40), (20, 9, 1032)])
@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("shared", [False, True])
def test_combine(rng, N, topk, M, type, shared):
    items = N * topk
    Y = cuda(rng.standard_normal((items, M)), type)
    pos = rng.permutation(items).reshape(N, topk).astype(np.int32)
    pos[rng.random((N, topk)) < 0.2] = -1
    weights = cuda(rng.random((N, topk)), "f32")
    weights[cuda(pos < 0)] = float("nan")                     # not looked at
    sh = cuda(rng.standard_normal((N, M)), "f32") if shared else None
    out = q6.moe_combine(Y, cuda(pos), weights, shared=sh)
    wt, y = np.where(pos < 0, 0, f64(weights)), f64(Y)[np.maximum(pos, 0)]
    terms = np.where((pos < 0)[..., None], 0, wt[..., None] * y)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    if shared:
        want, size = want + f64(sh), size + np.abs(f64(sh))
    u = ref.ROUND[type]
    check(out, want, u * np.abs(want) + (1 + u) * (topk + 2) * 2.0 ** -24 * size + 2.0 ** -25)


def test_combine_strided(rng):
    Y = cuda(rng.standard_normal((6, 80)), "bf16")[:, :72]
    pos = cuda(np.arange(6, dtype=np.int32).reshape(3, 2))
    weights = cuda(np.ones((3, 2)), "f32")
    out = torch.zeros((3, 75), dtype=torch.bfloat16, device="cuda")
    q6.moe_combine(Y, pos, weights, out=out[:, :72])
    assert torch.equal(out[:, :72], (Y[0::2].float() + Y[1::2].float()).bfloat16())
    assert not out[:, 72:].any()


# --------------------------------------------------------------------- lora ---

def run_lora(rng, N, L, r, K, M, xtype="f32", type="bf16", ids=None, in_place=False, pad=0):
    ids = rng.integers(-1, L, N) if ids is None else ids
    X = cuda(rng.standard_normal((N, K + pad)), xtype)[:, :K]
    A = cuda(rng.standard_normal((L, r, K)) / np.sqrt(K), type)
    B = cuda(rng.standard_normal((L, M, r)) / np.sqrt(r), type)
    scale = cuda(rng.standard_normal(L), "f32")
    Y = cuda(rng.standard_normal((N, M + pad)), "f32")[:, :M]
    want, bound = ref.lora(f64(Y), f64(X), f64(A), f64(B), f64(scale), ids)
    g = q6.group_rows(cuda(ids.astype(np.int32)), L)
    keep = Y.clone()
    ad = q6.LoraAdapters(A, B, scale)
    out = q6.lora_add(ad, X, g, Y, out=None if in_place else torch.empty_like(keep))
    assert (out is Y) == in_place
    check(out, want, bound)
    none = cuda(ids < 0)
    assert torch.equal(out[none], keep[none])


@pytest.mark.parametrize("N,L,r,K,M", [(1, 1, 8, 32, 1), (1, 4, 16, 4096, 512), (2, 3, 24, 96, 33),
                                       (47, 24, 32, 1024, 200), (100, 2, 64, 512, 130),
                                       (333, 5, 128, 1056, 97), (70, 70, 8, 256, 1001),
                                       (40, 1, 256, 288, 64), (65, 1, 72, 64, 300)])
@pytest.mark.parametrize("xtype,type", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"),
                                        ("f16", "bf16")])
def test_lora(rng, N, L, r, K, M, xtype, type):
    run_lora(rng, N, L, r, K, M, xtype, type)


@pytest.mark.parametrize("counts", [[16], [17, 0, 1], [0, 32, 33], [15, 16, 31, 100]])
def test_lora_group_sizes(rng, counts):
    ids = rng.permutation(np.concatenate([np.full(c, a) for a, c in enumerate(counts)]))
    run_lora(rng, len(ids), len(counts), 16, 256, 96, ids=ids)


def test_lora_in_place_and_strided(rng):
    run_lora(rng, 37, 3, 16, 512, 100, in_place=True)
    run_lora(rng, 37, 3, 16, 512, 100, pad=8)
    run_lora(rng, 120, 3, 16, 512, 101, in_place=True, pad=8)


def test_lora_no_token_has_one(rng):
    run_lora(rng, 9, 2, 8, 64, 40, ids=np.full(9, -1))


def test_lora_without_tokens():
    ad = q6.LoraAdapters(torch.zeros((2, 8, 64), device="cuda", dtype=torch.float16),
                         torch.zeros((2, 16, 8), device="cuda", dtype=torch.float16),
                         torch.ones(2, device="cuda"))
    g = q6.group_rows(torch.empty((0,), dtype=torch.int32, device="cuda"), 2)
    out = q6.lora_add(ad, torch.empty((0, 64), device="cuda"), g, torch.empty((0, 16), device="cuda"))
    assert out.shape == (0, 16)


# --------------------------------------------------- streams, graphs, errors ---

def moe_step(w_up, w_down, logits, X, topk):
    r = q6.moe_route(logits, topk)
    h, _ = q6.experts_mmq(w_up, X, r.groups)
    y, _ = q6.experts_mmq(w_down, h, r.groups, gather=False)
    return q6.moe_combine(y, r.groups.pos, r.weights)


@pytest.mark.parametrize("N", [3, 200])
def test_moe_step_on_a_side_stream_and_in_a_graph(rng, N):
    E, H, D, topk = 6, 64, 512, 2
    w_up = q6.pack_experts(cuda(raw_experts(1, "q4_K", E, 2 * 256, D)), "q4_K", E, 2 * 256, D,
                           swiglu=True)
    w_down = q6.pack_experts(cuda(raw_experts(2, "q6_K", E, D, 256)), "q6_K", E, D, 256)
    X = cuda(rng.standard_normal((N, D)) / 64, "bf16")
    logits = cuda(rng.standard_normal((N, E)), "f32")
    want = moe_step(w_up, w_down, logits, X, topk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = moe_step(w_up, w_down, logits, X, topk)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    x2, l2 = torch.zeros_like(X), torch.zeros_like(logits)
    with torch.cuda.graph(graph):
        out = moe_step(w_up, w_down, l2, x2, topk)
    x2.copy_(X)
    l2.copy_(logits)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_stream_argument(rng):
    """The stream argument, scratch memory included."""
    side = torch.cuda.Stream()
    ids = cuda(rng.integers(0, 3, 50).astype(np.int32))
    A = cuda(rng.standard_normal((3, 16, 256)), "f16")
    B = cuda(rng.standard_normal((3, 64, 16)), "f16")
    ad = q6.LoraAdapters(A, B, torch.ones(3, device="cuda"))
    X, Y = cuda(rng.standard_normal((50, 256)), "f32"), cuda(rng.standard_normal((50, 64)), "f32")
    want = q6.lora_add(ad, X, q6.group_rows(ids, 3), Y, out=torch.empty_like(Y))
    torch.cuda.synchronize()
    g = q6.group_rows(ids, 3, stream=side)
    got = q6.lora_add(ad, X, g, Y, out=torch.empty_like(Y), stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals(rng):
    X = cuda(rng.standard_normal((4, 512)), "bf16")
    w = q6.pack_experts(cuda(raw_experts(1, "q4_K", 2, 32, 512)), "q4_K", 2, 32, 512)
    g = q6.group_rows(cuda(np.zeros((4, 2), np.int32)), 2)
    bad = [lambda: q6.experts_mmq(w, X.float(), g), lambda: q6.experts_mmq(w, X[:, :256], g),
           lambda: q6.experts_mmq(w, X[:3], g), lambda: q6.experts_mmq(w, X, g, gather=False),
           lambda: q6.experts_mmq(w, X.cpu(), g),
           lambda: q6.experts_mmq(w, X, q6.group_rows(cuda(np.zeros((4, 2), np.int32)), 3)),
           lambda: q6.experts_mmq(w, X, g, out=torch.empty((8, 31), dtype=torch.bfloat16, device="cuda")),
           lambda: q6.experts_mmq(w, torch.zeros(4 * 513 + 1, dtype=torch.bfloat16,
                                                 device="cuda")[1:].view(4, 513)[:, :512], g),
           lambda: q6.moe_route(X.double(), 2), lambda: q6.moe_route(X, 33),
           lambda: q6.moe_route(X[:, :4], 5), lambda: q6.moe_route(X.t(), 2),
           lambda: q6.moe_route(X, 2, out=q6.alloc_route(4, 512, 3)),
           lambda: q6.group_rows(g.pos.long(), 2), lambda: q6.group_rows(g.pos, 1025),
           lambda: q6.pack_experts(torch.zeros(100, dtype=torch.uint8, device="cuda"), "q4_K", 1, 1, 256),
           lambda: q6.moe_combine(X, g.pos, torch.ones((4, 1), device="cuda")),
           lambda: q6.LoraAdapters(X.view(1, 4, 512), X.view(1, 512, 4), torch.ones(1, device="cuda")),
           lambda: q6.LoraAdapters(X.view(1, 4, 512).half(), X.view(1, 512, 4), torch.ones(1, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(q6.Q6Error):
            call()
            pytest.fail(f"call {i} was accepted")


@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_example_layer(tokens):
    """The example's layer against 64 bits. Its int8 activations dominate: a value's step is 1/127
    of its block's largest, about 3, so the rounding error is 3 / 127 / sqrt(12) of a unit value,
    0.7 %; the experts' part has bf16 activations (2^-9 each way) and results."""
    import importlib
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    assert importlib.import_module("moe_layer").check(tokens) <= 0.015


# ------------------------------------------------- offsets that pass 32 bits ---

@pytest.mark.parametrize("N", [2, 600])
def test_experts_plane_past_4_gib(rng, N):
    E, M, K = 40, 16384, 16384
    gen = torch.Generator("cuda").manual_seed(N)
    raw = torch.randint(0, 256, (E, M, K // 256, 144), generator=gen, device="cuda",
                        dtype=torch.uint8)
    d = torch.tensor([1e-4, 7e-4], device="cuda").half().view(torch.uint8)
    raw[..., 0:4] = d
    w = q6.pack_experts(raw, "q4_K", E, M, K)
    assert w.plane.numel() > 1 << 32
    rows = np.array([0, 1, 127, 128, 9000, M - 2, M - 1])
    some = raw[E - 1, torch.from_numpy(rows).cuda()].cpu().numpy().reshape(1, len(rows), -1)
    del raw
    X = cuda(rng.standard_normal((N, K)), "bf16")
    ids = np.full((N, 1), E - 1)
    Y, path = q6.experts_mmq(w, X, q6.group_rows(cuda(ids.astype(np.int32)), E))
    assert path == ("experts_few" if N == 2 else "experts_tc")
    q6.sync_status()
    want, bound = ref.experts(some, "q4_K", f64(X), np.zeros_like(ids), 1, False, True, "bf16")
    check(Y[:, torch.from_numpy(rows).cuda()], want, bound)


def test_combine_past_2_31_values():
    N, topk, M = 70000, 8, 4096
    Y = torch.zeros((N * topk, M), dtype=torch.bfloat16, device="cuda")
    assert Y.numel() > 1 << 31
    Y[-topk:] = torch.arange(1, topk + 1, device="cuda")[:, None]
    pos = torch.arange(N * topk, dtype=torch.int32, device="cuda").view(N, topk)
    out = q6.moe_combine(Y, pos, torch.ones((N, topk), device="cuda"))
    assert (out[-1] == 36).all() and not out[:-1].any()


def test_lora_past_2_31_values(rng):
    N, K, M, r = 140000, 16384, 24, 8
    X = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    assert X.numel() > 1 << 31
    last = cuda(rng.standard_normal((3, K)), "bf16")
    X[-3:] = last
    A, B = cuda(rng.standard_normal((2, r, K)) / 128, "bf16"), cuda(rng.standard_normal((2, M, r)), "bf16")
    scale, Y = torch.ones(2, device="cuda"), torch.zeros((N, M), device="cuda")
    ids = np.ones(N, np.int64)
    out = q6.lora_add(q6.LoraAdapters(A, B, scale), X, q6.group_rows(cuda(ids.astype(np.int32)), 2), Y)
    want, bound = ref.lora(np.zeros((3, M)), f64(last), f64(A), f64(B), f64(scale), ids[:3])
    check(out[-3:], want, bound)
    assert not out[:-3].any()


# --------------------------------------------------- calls one behind another ---

@pytest.mark.parametrize("type", ["bf16", "f16"])
def test_calls_follow_each_other(rng, type):
    """Calls in a row, whose kernels overlap (weights may be read while the rows of x are still
    made, B and Y while T is), give what they give with the device idle between them: every step
    has new weights in the memory of the last, new tokens and new groups."""
    E, M, K, L, r, N = 6, 520, 1024, 3, 16, 300
    raws = [cuda(raw_experts(20 + i, "q4_K", E, M, K)) for i in range(4)]
    Xs = [cuda(rng.standard_normal((N, K)), type) for _ in range(4)]
    lists = [cuda(rng.integers(-1, E, (N, 2)).astype(np.int32)) for _ in range(4)]
    own = [cuda(rng.integers(-1, L, (N,)).astype(np.int32)) for _ in range(4)]
    ABs = [(cuda(rng.standard_normal((L, r, K)), type), cuda(rng.standard_normal((L, M, r)), type))
           for _ in range(4)]
    scale = torch.ones(L, device="cuda")

    def steps(idle):
        wait = torch.cuda.synchronize if idle else (lambda: None)
        raw, X = torch.empty_like(raws[0]), torch.empty_like(Xs[0])
        A, B = torch.empty_like(ABs[0][0]), torch.empty_like(ABs[0][1])
        plane = None
        got = []
        for i in range(24):
            k = i * 5 % 4
            raw.copy_(raws[k]), X.copy_(Xs[(k + i) % 4])
            A.copy_(ABs[k][0]), B.copy_(ABs[k][1])
            wait()
            w = q6.pack_experts(raw, "q4_K", E, M, K)
            if plane is not None:
                plane.plane.copy_(w.plane)
                w = plane
            plane = w
            wait()
            g = q6.group_rows(lists[(i // 2) % 4], E)
            wait()
            Y, path = q6.experts_mmq(w, X, g)
            assert path == "experts_tc"
            wait()
            t = q6.moe_combine(Y, g.pos, torch.full((N, 2), 0.5, device="cuda")).float()
            wait()
            mine = q6.group_rows(own[i % 4], L)
            wait()
            out = q6.lora_add(q6.LoraAdapters(A, B, scale), X, mine, t)
            wait()
            got += [Y.clone(), out.clone()]
        q6.sync_status()
        return got

    for a, b in zip(steps(True), steps(False)):
        assert torch.equal(a, b)
