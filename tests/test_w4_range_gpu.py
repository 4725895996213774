"""Activations at the ends of their range through 4-bit weights, on a GB300: what the
header says of infinities and of large bf16 numbers where few rows stream the weights."""
import pytest

import dense_fp16_gemm_f16_gb300 as g
import llm_check as lc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


def _bound(A, W):
    w, mag = lc.w64(W)
    a = A.double()
    ref = a @ w.t()
    return ref, 1.01 * lc.U[A.dtype] * ref.abs() + lc.E32 * (a.abs() @ mag.t()) + lc.FLOOR


@pytest.mark.parametrize("M", [1, 8, 13, 16, 20])
@pytest.mark.parametrize("group,asym", [(32, True), (64, False), (128, True), (128, False)])
def test_bf16_up_to_2_to_the_113(M, group, asym):
    gen = torch.Generator().manual_seed(M + group)
    N, K = 136, 1024                                   # small: 20 rows stream the weights too
    A = (torch.rand((M, K), generator=gen) * 2 - 1) * 2.0 ** 113
    A[0] = 2.0 ** 113                                  # every element of a row, one sign
    A = A.bfloat16().cuda()
    W = lc.random_w4(gen, (), N, K, group, asym, A.dtype)
    D = torch.full((M, N), float("nan"), dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=D.device)
    lc.check(D, *_bound(A, W), "large numbers")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [2, 8, 16, 20])
@pytest.mark.parametrize("asym", [False, True])
def test_an_infinity_makes_its_row_nan(dtype, M, asym):
    gen = torch.Generator().manual_seed(M)
    N, K = 136, 1024
    A = torch.randn((M, K), generator=gen).to(TYPES[dtype]).cuda()
    W = lc.random_w4(gen, (), N, K, 64, asym, A.dtype)
    ref, tol = _bound(A, W)
    A[1, 77] = float("inf")
    D = torch.zeros((M, N), dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=D.device)
    assert bool(torch.isnan(D[1]).all())
    others = torch.arange(M, device="cuda") != 1
    lc.check(D[others], ref[others], tol[others], "other rows")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("where", ["first", "between"])
def test_an_infinity_makes_its_token_nan(dtype, where):
    gen = torch.Generator().manual_seed(5)
    T, H, I, E = 6, 256, 128, 2
    X = torch.randn((T, H), generator=gen).to(TYPES[dtype]).cuda()
    W13, W2 = (lc.random_w4(gen, (E,), rows, K, 64, False, X.dtype) for rows, K in ((2 * I, H), (H, I)))
    ids = (torch.arange(T, dtype=torch.int32) % E).view(T, 1).cuda()
    weights = torch.ones((T, 1), device="cuda")
    ref, tol = lc.ffn64(X, ids, weights, W13, W2)
    if where == "first":
        X[3, 9] = float("-inf")
    else:
        X[3] *= 1e3 if dtype == "f16" else 2.0 ** 70   # gate * up beyond the type's largest number
    Y = torch.zeros((T, H), dtype=X.dtype, device="cuda")
    g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
    g.gemm_f16_nt_check(device=Y.device)
    assert bool(torch.isnan(Y[3]).all())
    others = torch.arange(T, device="cuda") != 3
    lc.check(Y[others], ref[others], tol[others], "other tokens")
