"""Rows and stacks whose lengths pass what 32-bit byte counts hold, on a GB300.

Activations are zero but at both ends, so the 64-bit form needs only the weights
there; every weight is read all the same, and whatever is read from elsewhere shows."""
import pytest

import dense_fp16_gemm_f16_gb300 as g
import llm_check as lc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

END = 640   # elements at each end that are not zero, a multiple of every group


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def _rows(gen, n, K, dtype):
    """n rows of K, random at both ends and zero between."""
    A = torch.zeros((n, K), dtype=dtype, device="cuda")
    A[:, :END].normal_(generator=gen)
    A[:, -END:].normal_(generator=gen)
    return A


def _ends(t):
    return torch.cat((t[..., :END], t[..., -END:]), -1)


def _w4(gen, lead, N, K, group, dtype):
    return g.W4(torch.randint(0, 256, (*lead, N, K // 2), generator=gen, dtype=torch.uint8, device="cuda"),
                torch.rand((*lead, K // group, N), generator=gen, device="cuda", dtype=dtype) * 0.02 + 0.01, None, group)


def _w4_ends(W):
    """The same rows, only the k at both ends."""
    half, groups = END // 2, END // W.group
    return g.W4(torch.cat((W.codes[..., :half], W.codes[..., -half:]), -1),
                torch.cat((W.scales[..., :groups, :], W.scales[..., -groups:, :]), -2), None, W.group)


def _one_expert(H, I, group):
    """One token through one expert with 4-bit first and 16-bit second weights of H x I."""
    gen = torch.Generator(device="cuda").manual_seed(H % 1000)
    dtype = torch.bfloat16
    X = _rows(gen, 1, H, dtype)
    W13 = _w4(gen, (1,), 2 * I, H, group, dtype)
    W2 = torch.randn((1, H, I), generator=gen, device="cuda", dtype=dtype)
    ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    weights = torch.ones((1, 1), device="cuda")
    Y = torch.full_like(X, float("nan"))
    g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
    g.gemm_f16_nt_check(device=X.device)
    # the form of the few columns that count, its outputs at both ends, and the middle by slices
    small = _w4_ends(W13)
    wide = torch.cat((W2[:, :END], W2[:, -END:]), 1)
    lc.check(_ends(Y), *lc.ffn64(_ends(X), ids, weights, small, wide), f"H = {H}, ends")
    a, _ = lc.w64(g.W4(small.codes[0], small.scales[0], None, group))
    gu = _ends(X).double() @ a.t()
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    step = 1 << 26
    for r in range(0, H, step):
        ref = (W2[0, r:r + step].double() * h).sum(-1)
        # loose: this finds outputs that are missing or of other rows
        assert bool(((Y[:, r:r + step].double() - ref).abs() <= 0.02 * ref.abs() + 1e-3 * h.norm()).all())


def test_experts_with_columns_past_two_gigabytes():
    # eight columns of H pass 2^31 bytes: they do not fit shared memory, whatever 32 bits say
    _one_expert(1 << 27, 8, 128)


def test_router_with_the_longest_rows():
    H, E = 2 ** 31 - 8, 2
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.zeros((1, H), dtype=torch.float16, device="cuda")
    Wr = torch.ones((E, H), dtype=torch.float16, device="cuda")
    for part in (slice(0, 64), slice(H - 64, H)):
        X[:, part] = torch.randint(-2, 3, (1, 64), generator=gen, device="cuda").half()
        Wr[:, part] = torch.randint(-2, 3, (E, 64), generator=gen, device="cuda").half()
    ids, w = g.gemm_moe_route(X, Wr, k=E)
    g.gemm_f16_nt_check(device=X.device)
    x, r = (torch.cat((t[:, :64], t[:, -64:]), 1) for t in (X, Wr))
    rid, rw = lc.route64(x, r, E)
    assert torch.equal(ids, rid)
    assert bool(((w.double() - rw).abs() <= 2.0 ** -19 * rw + 1e-37).all())


def test_router_with_many_tokens():
    # more tokens than have their logits in scratch at one time, and a few left over
    T, H, E, k = 16389, 72, 40, 3
    gen = torch.Generator().manual_seed(6)
    X = torch.randint(-1, 2, (T, H), generator=gen).bfloat16().cuda()
    Wr = torch.randint(-1, 2, (E, H), generator=gen).bfloat16().cuda()
    ids, w = g.gemm_moe_route(X, Wr, k=k)
    rid, rw = lc.route64(X, Wr, k)
    assert torch.equal(ids, rid)
    assert bool(((w.double() - rw).abs() <= 2.0 ** -19 * rw + 1e-37).all())


def test_product_with_the_longest_rows():
    N, K, group = 16, 2 ** 31 - 128, 128
    gen = torch.Generator(device="cuda").manual_seed(7)
    A = _rows(gen, 1, K, torch.float16)
    W = _w4(gen, (), N, K, group, torch.float16)
    D = torch.full((1, N), float("nan"), dtype=torch.float16, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=D.device)
    w, mag = lc.w64(_w4_ends(W))
    a = _ends(A).double()
    ref = a @ w.t()
    lc.check(D, ref, 1.01 * lc.U[D.dtype] * ref.abs() + lc.E32 * (a.abs() @ mag.t()) + lc.FLOOR, f"K = {K}")


@pytest.mark.parametrize("M", [1, 17])
def test_product_with_the_most_rows_of_weights(M):
    N, K, group = 2 ** 31 - 8, 32, 32
    gen = torch.Generator(device="cuda").manual_seed(8)
    A = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    W = _w4(gen, (), N, K, group, torch.bfloat16)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=D.device)
    # nothing is left out, and slices in fp32: exact to 2^-20 of the sums' magnitudes
    step, worst = 1 << 22, 0.0
    assert not any(bool(torch.isnan(D[m]).any()) for m in range(M))
    for r in (0, 1 << 29, (1 << 30) - step // 2, 3 << 29, N - step):
        w, _ = lc.w64(g.W4(W.codes[r:r + step], W.scales[:, r:r + step], None, group))
        w = w.float()
        d = D[:, r:r + step].float()
        for m in range(M):
            prod = w * A[m].float()
            ref = prod.sum(1)
            off = (d[m] - ref).abs() - 1.01 * lc.U[D.dtype] * ref.abs()
            # offset codes enter the sums: see llm_check
            worst = max(worst, float((off / (prod.abs().sum(1) + 4 * A[m].float().abs().sum())).max()))
    assert worst <= 2.0 ** -20


def test_experts_with_the_longest_rows():
    _one_expert(2 ** 31 - 128, 8, 128)
