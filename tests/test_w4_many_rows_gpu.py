"""The 4-bit product with a prompt's rows on a GB300, against the 64-bit form."""
import pytest

import dense_fp16_gemm_f16_gb300 as g
import llm_check as lc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,group,asym", [(1000, 1000, 1056, 32, True), (4099, 264, 512, 64, False),
                                              (2048, 2048, 2048, 128, True), (8192, 136, 384, 128, False)])
def test_product(dtype, M, N, K, group, asym):
    gen = torch.Generator().manual_seed(M)
    A = torch.randn((M, K), generator=gen).to(dtype).cuda()
    W = lc.random_w4(gen, (), N, K, group, asym, dtype)
    D = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=D.device)
    w, mag = lc.w64(W)
    a = A.double()
    ref = a @ w.t()
    # the output's rounding, fp32 sums, and weights rounded to the type: 6 standard deviations of that many roundings
    tol = (1.01 * lc.U[dtype] * ref.abs() + lc.E32 * (a.abs() @ mag.t()) + lc.FLOOR
           + 6 * lc.U[dtype] * ((a * a) @ (w * w).t()).sqrt())
    lc.check(D, ref, tol, f"{M}x{N}x{K}")
