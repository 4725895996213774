"""Routing and the mixture-of-experts layer on a GB300 against plain 64-bit forms."""
import pytest

import dense_fp16_gemm_f16_gb300 as g
import llm_check as lc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------- routing
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scoring", list(g.MoeScoring))
@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (1, 2048, 64, 6), (3, 72, 8, 8), (64, 512, 256, 8), (17, 1000, 130, 16),
                                     (65, 264, 33, 3), (300, 64, 1024, 4), (8, 8192, 128, 2)])
def test_route_of_whole_numbers_is_exact(dtype, scoring, T, H, E, k):
    """Whole logits, exact in any order of summation, with many equal ones: the lower expert comes first."""
    gen = _gen(T + H + E)
    X = torch.randint(-1, 2, (T, H), generator=gen).to(TYPES[dtype]).cuda()
    Wr = (torch.randint(-1, 2, (E, H), generator=gen) * (torch.rand((E, H), generator=gen) < 8 / H)).to(X.dtype).cuda()
    for renormalize in (True, False):
        ids, w = g.gemm_moe_route(X, Wr, k=k, scoring=scoring, renormalize=renormalize)
        rid, rw = lc.route64(X, Wr, k, None, int(scoring), renormalize)
        assert torch.equal(ids, rid)
        # exp in fp32 (2 ulp and its argument's rounding), a sum over E and two divisions: 2^-19 covers them
        assert bool(((w.double() - rw).abs() <= 2.0 ** -19 * rw + 1e-37).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scoring", list(g.MoeScoring))
@pytest.mark.parametrize("T,H,E,k", [(1, 4096, 64, 4), (40, 1032, 96, 5), (64, 8192, 256, 8)])
def test_route_weights(dtype, scoring, T, H, E, k):
    gen = _gen(T + E)
    X = torch.randn((T, H), generator=gen).to(TYPES[dtype]).cuda()
    Wr = (torch.randn((E, H), generator=gen) * 1.5 / H ** 0.5).to(X.dtype).cuda()
    bias = (torch.randn(E, generator=gen) * 0.1).cuda()
    mag = (X.double().abs() @ Wr.double().abs().t()).amax()
    delta = float(2 * lc.E32 * mag)               # how far a logit may be off
    for b in (None, bias):
        logits = X.double() @ Wr.double().t()
        p = torch.softmax(logits, 1) if scoring == 0 else torch.sigmoid(logits)
        key = logits if b is None else p + b.double()
        ids, w = g.gemm_moe_route(X, Wr, k=k, bias=b, scoring=scoring)
        rid, rw = lc.route64(X, Wr, k, b, int(scoring))
        # an order that hangs on less than the bound may go either way
        gaps = key.sort(1, descending=True).values
        clear = ((gaps[:, :k] - gaps[:, 1:k + 1]) > 2 * delta).all(1)
        assert float(clear.float().mean()) > 0.5
        assert torch.equal(ids[clear], rid[clear])
        assert bool(((w.double() - rw)[clear].abs() <= (4 * delta + 2.0 ** -19) * rw[clear]).all())


def test_route_masks_and_values_that_are_not_numbers():
    T, H, E, k = 6, 64, 40, 4
    gen = _gen(9)
    X = torch.randint(-2, 3, (T, H), generator=gen).half().cuda()
    Wr = torch.randint(-2, 3, (E, H), generator=gen).half().cuda()
    bias = torch.zeros(E, device="cuda")
    bias[::2] = -INF
    for scoring in g.MoeScoring:
        # a sigmoid saturates to equal scores in fp32 well before it does in 64 bits: keep the logits small
        x = X if scoring == 0 else (X / 32)
        ids, w = g.gemm_moe_route(x, Wr, k=k, bias=bias, scoring=scoring)
        assert bool((ids % 2 == 1).all()) and bool((ids >= 0).all())
        bias3 = torch.full((E,), -INF, device="cuda")
        bias3[[3, 11]] = 0.0
        ids, w = g.gemm_moe_route(x, Wr, k=k, bias=bias3, scoring=scoring)
        rid, rw = lc.route64(x, Wr, k, bias3, int(scoring))
        assert bool((ids[:, 2:] == -1).all()) and bool((w[:, 2:] == 0).all())
        assert torch.equal(ids[:, :2].sort(1).values, torch.tensor([[3, 11]], device="cuda", dtype=torch.int32).expand(T, 2))
        assert bool(((w.sum(1) - 1).abs() < 1e-6).all())
        ids, w = g.gemm_moe_route(x, Wr, k=k, bias=torch.full((E,), -INF, device="cuda"), scoring=scoring)
        assert bool((ids == -1).all()) and bool((w == 0).all())
    # the type's lowest value as a mask: still chosen when nothing else is left, in order
    low = torch.full((E,), torch.finfo(torch.float32).min, device="cuda")
    low[7] = 0.0
    ids, w = g.gemm_moe_route(X, Wr, k=3, bias=low)
    assert ids[:, 0].tolist() == [7] * T and ids[:, 1].tolist() == [0] * T and ids[:, 2].tolist() == [1] * T
    # a token of NaN chooses nothing and leaves the others alone
    clean = g.gemm_moe_route(X, Wr, k=k)
    X[2] = float("nan")
    ids, w = g.gemm_moe_route(X, Wr, k=k)
    assert bool((ids[2] == -1).all()) and bool((w[2] == 0).all())
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(ids[keep], clean[0][keep]) and torch.equal(w[keep], clean[1][keep])


# ------------------------------------------------------------- the experts
def _experts(gen, E, H, I, dtype, kind13, kind2):
    def one(rows, K, kind):
        if kind == 0:
            return (torch.randn((E, rows, K), generator=gen) / K ** 0.5).to(dtype).cuda()
        return lc.random_w4(gen, (E,), rows, K, abs(kind), kind < 0, dtype)
    return one(2 * I, H, kind13), one(H, I, kind2)


# kinds: 0 = 16-bit, a group = 4-bit symmetric, minus a group = 4-bit with zero points
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I,E,k,kind13,kind2", [
    (1, 8, 8, 1, 1, 0, 0), (1, 2048, 1024, 16, 6, 0, 0), (2, 520, 264, 4, 2, 0, 0), (5, 1032, 200, 6, 3, 0, 0),
    (9, 256, 1000, 3, 3, 0, 0), (33, 512, 384, 8, 2, 0, 0), (64, 384, 136, 64, 8, 0, 0), (64, 264, 72, 2, 2, 0, 0),
    (1, 256, 128, 4, 2, 128, 128), (3, 288, 96, 5, 2, -32, 32), (8, 512, 192, 16, 4, 64, -64),
    (17, 640, 384, 8, 2, -128, 128), (64, 256, 320, 32, 8, 32, 64), (64, 128, 128, 2, 1, 128, -128),
    (12, 384, 256, 4, 2, 0, -32), (12, 384, 256, 4, 2, 64, 0), (40, 1024, 704, 24, 6, 64, 64)])
def test_ffn(dtype, T, H, I, E, k, kind13, kind2):
    gen = _gen(T + H + I + E)
    X = torch.randn((T, H), generator=gen).to(TYPES[dtype]).cuda()
    W13, W2 = _experts(gen, E, H, I, X.dtype, kind13, kind2)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32).cuda()
    weights = torch.rand((T, k), generator=gen).cuda()
    Y = torch.full((T, H), float("nan"), dtype=X.dtype, device="cuda")
    g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
    g.gemm_f16_nt_check(device=X.device)
    lc.check(Y, *lc.ffn64(X, ids, weights, W13, W2), "ffn")
    again = torch.empty_like(Y)
    g.gemm_moe_ffn(X, ids, weights, W13, W2, again)
    assert torch.equal(Y, again)


@pytest.mark.parametrize("kind", [0, -32])
@pytest.mark.parametrize("T", [1, 7, 64])
def test_ffn_of_odd_choices(T, kind):
    """Ids outside the experts, experts listed twice, tokens with no expert, all tokens on one expert."""
    H, I, E, k = 288, 160, 6, 4
    gen = _gen(T)
    X = torch.randn((T, H), generator=gen).bfloat16().cuda()
    W13, W2 = _experts(gen, E, H, I, X.dtype, kind, kind)
    weights = torch.randn((T, k), generator=gen).cuda()
    for ids in (torch.randint(-2, E + 2, (T, k), generator=gen), torch.full((T, k), 5), torch.full((T, k), -1),
                torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 0]).expand(T, 4), torch.tensor([1, -1, 1, 3]).expand(T, 4)):
        ids = ids.to(torch.int32).contiguous().cuda()
        Y = torch.full((T, H), float("nan"), dtype=X.dtype, device="cuda")
        g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
        g.gemm_f16_nt_check(device=X.device)
        lc.check(Y, *lc.ffn64(X, ids, weights, W13, W2), "ffn")
        none = ((ids < 0) | (ids >= E)).all(1)
        assert bool((Y[none] == 0).all())


@pytest.mark.parametrize("kind", [0, 64])
def test_ffn_keeps_values_that_are_not_finite_apart(kind):
    T, H, I, E, k = 10, 320, 192, 5, 2
    gen = _gen(4)
    X = torch.randn((T, H), generator=gen).half().cuda()
    W13, W2 = _experts(gen, E, H, I, X.dtype, kind, kind)
    ids = torch.randint(0, 3, (T, 1), generator=gen)
    ids = torch.cat((ids, ids + 1), 1).to(torch.int32).cuda()         # experts 0..3; expert 4 is not chosen
    weights = torch.rand((T, k), generator=gen).cuda()
    ref, tol = lc.ffn64(X, ids, weights, W13, W2)
    for w in (W13, W2):
        (w if kind == 0 else w.scales)[4].fill_(float("nan"))
    X[3, 5], X[7] = INF, float("nan")
    Y = torch.full((T, H), float("nan"), dtype=X.dtype, device="cuda")
    g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[3, 7]] = False
    assert not bool(torch.isfinite(Y[~keep]).any())
    lc.check(Y[keep], ref[keep], tol[keep], "other tokens")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I,E,k,kind", [(1, 1024, 512, 32, 4, 0), (20, 512, 256, 8, 2, 128), (64, 256, 192, 64, 8, 64)])
def test_layer_is_route_then_ffn(dtype, T, H, I, E, k, kind):
    gen = _gen(T + E)
    X = torch.randn((T, H), generator=gen).to(TYPES[dtype]).cuda()
    Wr = torch.randn((E, H), generator=gen).to(X.dtype).cuda() / 16
    bias = (torch.randn(E, generator=gen) * 0.1).cuda()
    W13, W2 = _experts(gen, E, H, I, X.dtype, kind, kind)
    for scoring, b, renormalize in ((g.MoeScoring.SOFTMAX, None, True), (g.MoeScoring.SIGMOID, bias, False)):
        ids, weights = g.gemm_moe_route(X, Wr, k=k, bias=b, scoring=scoring, renormalize=renormalize)
        Y, Z = (torch.full((T, H), float("nan"), dtype=X.dtype, device="cuda") for _ in range(2))
        g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
        g.gemm_moe_layer(X, Wr, W13, W2, Z, k, bias=b, scoring=scoring, renormalize=renormalize)
        g.gemm_f16_nt_check(device=X.device)
        assert torch.equal(Y, Z)
        lc.check(Z, *lc.ffn64(X, ids, weights, W13, W2), "layer")


def test_layers_in_a_row_streams_and_graph():
    """Layers of different sizes one behind the other on one stream, on two streams at once, and from a graph."""
    cases = []
    for i, (T, H, I, E, k, kind) in enumerate([(4, 512, 256, 8, 2, 0), (64, 256, 384, 16, 4, 64), (1, 1024, 128, 4, 1, 0)]):
        gen = _gen(i)
        X = torch.randn((T, H), generator=gen).half().cuda()
        Wr = (torch.randn((E, H), generator=gen) / 16).half().cuda()
        W13, W2 = _experts(gen, E, H, I, X.dtype, kind, kind)
        Y = torch.empty_like(X)
        g.gemm_moe_layer(X, Wr, W13, W2, Y, k)
        torch.cuda.synchronize()
        cases.append((X, Wr, W13, W2, k, Y.clone()))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for rep in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                for X, Wr, W13, W2, k, ref in cases:
                    Y = torch.empty_like(X)
                    g.gemm_moe_layer(X, Wr, W13, W2, Y, k)
                    outs.append((Y, ref))
    torch.cuda.synchronize()
    assert all(torch.equal(Y, ref) for Y, ref in outs)
    s = streams[0]
    ys = [torch.empty_like(c[0]) for c in cases]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for (X, Wr, W13, W2, k, _), Y in zip(cases, ys):
            g.gemm_moe_layer(X, Wr, W13, W2, Y, k, stream=s)
    for _ in range(2):
        for Y in ys:
            Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(Y, c[5]) for Y, c in zip(ys, cases))


def test_refusals():
    X = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    Wr = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    W13 = torch.zeros((8, 64, 64), dtype=torch.float16, device="cuda")
    W2 = torch.zeros((8, 64, 32), dtype=torch.float16, device="cuda")
    Y = torch.zeros_like(X)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    S = g.Status
    with pytest.raises(ValueError):
        g.gemm_moe_route(X, Wr)                                   # neither k nor ids
    with pytest.raises(TypeError):
        g.gemm_moe_route(X, Wr, ids.long(), w)
    with pytest.raises(g.GemmError) as e:
        g.gemm_moe_route(X, Wr, k=9)                              # more choices than experts
    assert e.value.status == S.ERR_INVALID_VALUE
    with pytest.raises(g.GemmError):
        g.gemm_moe_route(torch.zeros((4, 64), device="cuda").half(), torch.zeros((32, 64), device="cuda").half(), k=17)
    with pytest.raises(TypeError):
        g.gemm_moe_ffn(X, ids, w, W13.bfloat16(), W2, Y)
    with pytest.raises(ValueError):
        g.gemm_moe_ffn(X, ids, w, W13, W2[:7], Y)
    with pytest.raises(ValueError):
        g.gemm_moe_ffn(X, ids, w, W13[:, :63].contiguous(), W2, Y)
    with pytest.raises(g.GemmError) as e:
        g.gemm_moe_ffn(X, ids, w, W13, W2, X)                     # Y over X
    assert e.value.status == S.ERR_INVALID_VALUE
    many = torch.zeros((65, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(g.GemmError) as e:
        g.gemm_moe_layer(many, Wr, W13, W2, torch.zeros_like(many), 2)
    assert e.value.status == S.ERR_INVALID_VALUE
    none = torch.zeros((0, 64), dtype=torch.float16, device="cuda")
    g.gemm_moe_layer(none, Wr, W13, W2, none.clone(), 2)          # no tokens: nothing to do
