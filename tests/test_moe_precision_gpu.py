"""How exact the experts' h = silu(gate) * up is where the sigmoid is far from one, on a GB300."""
import pytest

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


def test_h_keeps_its_precision_for_gates_far_below_zero():
    """One token, one expert.  Output r is 2^12 (h_r + c_r), h_r the h of a gate between -26 and -22 and c_r the
    fp16 number nearest to -h_r, itself an h: that of a gate of 32, whose silu is 32 in fp32.  What is left is
    what h_r holds beyond fp16.  Every sum of either product has one term, or two that cancel exactly, so the
    bound is that of h alone: exp 2 ulp (2^-22), the sum, the quotient and the product 2^-24 each, and the second
    part of h to half of fp16's smallest number, 2^-25; the output is then rounded to fp16."""
    gates = (torch.arange(-26 * 64, -22 * 64, dtype=torch.float64) / 64)          # fp16 numbers
    n = len(gates)
    silu = gates / (1 + torch.exp(-gates))
    factor = (-0.4 / silu / 2 ** 15).clamp(max=65504).half().double()              # up = factor * 2^15
    h = silu * factor * 2 ** 15
    assert bool((h < -0.25).all()) and bool((h > -0.5).all())
    c = (-h).half().double()
    H, I = n, 2 * n
    X = torch.zeros((1, H))
    X[0, 0], X[0, 1] = 2.0 ** 15, 1.0
    W13 = torch.zeros((1, 2 * I, H), dtype=torch.float64)
    r = torch.arange(n)
    W13[0, 2 * r, 1] = gates
    W13[0, I + 2 * r, 0] = factor
    W13[0, 2 * r + 1, 1] = 32.0
    W13[0, I + 2 * r + 1, 1] = c / 32
    W2 = torch.zeros((1, H, I), dtype=torch.float64)
    W2[0, r, 2 * r] = 2.0 ** 12
    W2[0, r, 2 * r + 1] = 2.0 ** 12
    for w in (W13, W2):
        assert torch.equal(w.half().double(), w)
    Y = torch.full((1, H), float("nan"), dtype=torch.float16, device="cuda")
    g.gemm_moe_ffn(X.half().cuda(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                   torch.ones((1, 1), device="cuda"), W13.half().cuda(), W2.half().cuda(), Y)
    g.gemm_f16_nt_check(device=Y.device)
    ref = 2.0 ** 12 * (h + c)
    tol = 2.0 ** 12 * (h.abs() * (2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -25) + 1.01 * 2.0 ** -11 * ref.abs() + 2.0 ** -25
    off = (Y[0].double().cpu() - ref).abs()
    assert bool((off <= tol).all()), f"{int((off > tol).sum())} of {n} out of bounds, worst {float((off / tol).max())} times"
