"""8-bit products with a scale per row of A, against 64 bits.

Bound per element, fixed before any run: one rounding of D (2^-8 of it for bf16, 1 %
wider), and fp32 sums of K products of 32 at a time whose K/32 additions, the two scales,
alpha, beta C and the bias are each off by at most 2^-23 of the magnitudes that enter.
"""
import pytest
import torch

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def draw(M, N, K, kind, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    top = 448.0 if kind == torch.float8_e4m3fn else 57344.0
    A, B = ((torch.randn(n, K, generator=gen, device=DEV) * top / 5).clamp(-top, top).to(kind) for n in (M, N))
    sm, sn = (torch.exp2(torch.rand(n, generator=gen, device=DEV) * 12 - 6) / top for n in (M, N))
    return A, B, sm, sn, gen


def check(D, A, B, sm, sn=None, alpha=1.0, beta=0.0, C=None, bias=None, relu=False):
    K = A.shape[1]
    f = alpha * sm.double()[:, None] * (1.0 if sn is None else sn.double()[None])
    a, b = A.float().double(), B.float().double()
    ref, mag = (a @ b.T) * f, (a.abs() @ b.abs().T) * f.abs()
    if C is not None:
        ref, mag = ref + beta * C.double(), mag + abs(beta) * C.double().abs()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    if relu:
        ref = ref.clamp(min=0)
    tol = 1.01 * 2.0 ** -8 * ref.abs() + (K / 32 + 6) * 2.0 ** -23 * mag
    bad = ~((D.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())


# every kernel that AUTO picks: column ranges with one CTA or a cluster each, for 16, 32
# and 64 rows; pieces of 128 x 256 tiles; split K over CTAs and over pairs; pairs; 512 x 256 tiles
SIZES = [(1, 8, 16), (3, 2048, 2048), (16, 520, 4096), (17, 8192, 1040), (33, 1000, 2064), (64, 8192, 512), (64, 136, 8192),
         (65, 72, 48), (200, 1000, 1040), (256, 256, 8192), (512, 2048, 8192), (128, 512, 16384), (700, 3000, 2048),
         (2048, 4104, 2048), (4100, 8200, 2064), (2304, 9000, 1024)]


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_rows_and_columns(M, N, K, kind):
    A, B, sm, sn, gen = draw(M, N, K, kind, M + N + K)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    g.gemm_nt_ex(A, B, D, scale_m=sm, scale_n=sn)
    check(D, A, B, sm, sn)
    C, bias = (torch.randn(s, generator=gen, device=DEV).bfloat16() for s in ((M, N), (N,)))
    E = C.clone()
    g.gemm_nt_ex(A, B, E, scale_m=sm, scale_n=sn, alpha=0.7, beta=-1.3, C=E, bias=bias, activation=g.Activation.RELU)
    check(E, A, B, sm, sn, 0.7, -1.3, C, bias, True)
    g.gemm_nt_ex(A, B, D, scale_m=sm)
    check(D, A, B, sm)
    g.gemm_f16_nt_check(device=DEV)


@pytest.mark.parametrize("M", [5, 300, 3000])
def test_scales_of_one_change_nothing(M):
    """With every row scale 1 the result is the plain product's, bit for bit."""
    A, B, _, sn, _ = draw(M, 4096, 2048, torch.float8_e4m3fn, M)
    D, E = (torch.empty(M, 4096, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gemm_nt_ex(A, B, D, scale_n=sn)
    g.gemm_nt_ex(A, B, E, scale_n=sn, scale_m=torch.ones(M, device=DEV))
    assert torch.equal(D, E)


def test_zero_and_nan_scales_stay_in_their_rows():
    for M in (4, 70):
        A, B, sm, sn, _ = draw(M, 256, 512, torch.float8_e4m3fn, 1)
        sm[1], sm[2] = 0.0, float("nan")
        D = torch.empty(M, 256, dtype=torch.bfloat16, device=DEV)
        g.gemm_nt_ex(A, B, D, scale_m=sm, scale_n=sn)
        keep = torch.tensor([i for i in range(M) if i != 2], device=DEV)
        check(D[keep], A[keep], B, sm[keep], sn)
        assert not bool(D[1].any()) and bool(D[2].isnan().all())


def test_a_part_of_a_batch():
    for first, last in ((1, 9), (3, 200)):
        A, B, sm, sn, _ = draw(last, 264, 512, torch.float8_e4m3fn, last)
        D = torch.empty(last - first, 264, dtype=torch.bfloat16, device=DEV)
        g.gemm_nt_ex(A[first:], B, D, scale_m=sm[first:], scale_n=sn)
        check(D, A[first:], B, sm[first:], sn)


def test_empty_sum():
    A, B = (torch.empty(n, 0, dtype=torch.float8_e4m3fn, device=DEV) for n in (3, 16))
    D = torch.full((3, 16), 9.0, dtype=torch.bfloat16, device=DEV)
    bias = torch.arange(16, device=DEV).bfloat16()
    g.gemm_nt_ex(A, B, D, scale_m=torch.full((3,), float("nan"), device=DEV), bias=bias)
    assert torch.equal(D, bias.expand(3, 16))


def test_after_the_norm_in_a_graph():
    """Norm, 8-bit rows, product: captured together and replayed on other activations."""
    for T in (3, 200):
        gen = torch.Generator(device=DEV).manual_seed(T)
        x = torch.randn(T, 2048, generator=gen, device=DEV).bfloat16()
        _, B, _, sn, _ = draw(1, 1024, 2048, torch.float8_e4m3fn, T)
        out = g.gemm_rmsnorm(x, Y8=g.Dtype.E4M3)
        D = torch.empty(T, 1024, dtype=torch.bfloat16, device=DEV)
        g.gemm_nt_ex(out.Y8, B, D, scale_m=out.scales, scale_n=sn)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.gemm_rmsnorm(x, Y8=out.Y8, scales=out.scales)
            g.gemm_nt_ex(out.Y8, B, D, scale_m=out.scales, scale_n=sn)
        for _ in range(3):
            x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
            graph.replay()
        torch.cuda.synchronize()
        check(D, out.Y8, B, out.scales, sn)
        h = x.double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
        assert bool(((out.Y8.float().double() * out.scales.double()[:, None] - y).abs() <= 0.07 * y.abs() + 2.0 ** -10 * 8).all())


def test_refusals():
    A, B, sm, sn, _ = draw(4, 64, 64, torch.float8_e4m3fn, 1)
    D = torch.empty(4, 64, dtype=torch.bfloat16, device=DEV)
    for error, change in [(TypeError, dict(scale_m=sm.double())), (ValueError, dict(scale_m=sm[:3])),
                          (ValueError, dict(scale_m=sm.cpu())), (ValueError, dict(variant=g.Variant.SKINNY_SPLITK))]:
        with pytest.raises(error):
            g.gemm_nt_ex(A, B, D, **(dict(scale_m=sm) | change))
    U = torch.empty(4, 64, dtype=torch.bfloat16, device=DEV)
    g.gemm_nt_ex(A.view(torch.uint8), B.view(torch.uint8), U, dtype=g.Dtype.E4M3, scale_m=sm)
    g.gemm_nt_ex(A, B, D, 4, 64, 64, scale_m=sm)
    assert torch.equal(U, D)
    g.gemm_nt_ex(A.data_ptr(), B.data_ptr(), U.zero_().data_ptr(), 4, 64, 64, dtype=g.Dtype.E4M3, scale_m=sm.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(U, D)
    for error, args, change in [(ValueError, (A, B, D, 5), {}), (TypeError, (A, B, D), dict(dtype=g.Dtype.E5M2)),
                                (TypeError, (A.view(torch.uint8), B.view(torch.uint8), D), {}),
                                (TypeError, (A, B, D.half()), {})]:
        with pytest.raises(error):
            g.gemm_nt_ex(*args, **(dict(scale_m=sm) | change))
    with pytest.raises(TypeError):
        H = A.float().half()
        g.gemm_nt_ex(H, H, torch.empty(4, 4, dtype=torch.float16, device=DEV), scale_m=sm)
