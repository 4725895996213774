"""4-bit weights on a GB300: packing, unpacking and the product D = A·Bᵀ
against plain 64-bit forms."""
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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------- packing
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("shape,group", [((8, 32), 32), ((24, 192), 64), ((40, 384), 128), ((3, 16, 96), 32),
                                         ((2, 1000, 1152), 128)])
def test_quantize_is_the_definition(dtype, asym, shape, group):
    W = torch.randn(shape, generator=_gen(sum(shape) + group)).to(TYPES[dtype])
    flat = W.view(-1, group)
    flat[0] = 0                                   # a group of zeros
    flat[1] = flat[1].abs()                       # no negative weight
    flat[2 % len(flat)] *= 1e-7                   # a scale that is tiny, in fp16 zero
    flat[3 % len(flat), 0] = 6e4                  # one weight far from the others
    W = W.cuda()
    out = g.gemm_w4_quantize(W, group, symmetric=not asym)
    codes, scales, zeros = lc.quantize64(W, group, asym)
    assert torch.equal(out.scales, scales.contiguous())
    assert torch.equal(out.codes, codes)
    assert (out.zeros is None) == (zeros is None)
    if asym:
        assert torch.equal(out.zeros, zeros.contiguous())
    values = g.gemm_w4_dequantize(out)
    assert torch.equal(values, lc.w64(out)[0].float().to(W.dtype))
    # half a step of error where the codes do not clip; a clipped one is off by the scale's own rounding
    step = out.scales.double().transpose(-1, -2).repeat_interleave(group, -1)
    lim = step * 0.51 + 15 * lc.U[W.dtype] * step + lc.U[W.dtype] * W.double().abs() + 8 * 2.0 ** -24
    assert bool(((values.double() - W.double()).abs() <= lim).all())


def test_exact_half_steps_go_to_the_even_code():
    # scale 1 exactly (largest magnitude 7), weights on half steps
    row = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 6.5] * 4)
    W = row.repeat(8, 1).half().cuda()
    out = g.gemm_w4_quantize(W, 32)
    assert torch.equal(out.scales, torch.ones_like(out.scales))
    want = torch.tensor([7.0, 0, 2, 2, 0, -2, -2, 6] * 4).half().cuda()
    assert torch.equal(g.gemm_w4_dequantize(out)[3], want)


def test_dequantize_takes_any_scales_and_zero_points():
    for dtype in TYPES.values():
        W = lc.random_w4(_gen(5), (2,), 24, 320, 64, True, dtype)
        assert torch.equal(g.gemm_w4_dequantize(W), lc.w64(W)[0].float().to(dtype))


def test_packing_nothing():
    out = g.gemm_w4_quantize(torch.empty((0, 64), dtype=torch.float16, device="cuda"), 32)
    assert g.gemm_w4_dequantize(out).shape == (0, 64)


# ------------------------------------------------------------- the product
def _product_ref(A, W, scale=1.0):
    w, mag = lc.w64(W)
    a = A.double()
    ref = a @ w.t()
    tol = 1.01 * lc.U[A.dtype] * ref.abs() + lc.E32 * (a.abs() @ mag.t()) + lc.FLOOR
    if A.shape[0] > 64:   # weights rounded to the type first: 6 standard deviations of that many roundings
        tol = tol + 6 * lc.U[A.dtype] * ((a * a) @ (w * w).t()).sqrt()
    return ref, tol


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("N,K,group", [(8, 32, 32), (24, 128, 128), (1000, 4128, 32), (2440, 192, 64), (776, 2944, 128)])
def test_product(dtype, asym, M, N, K, group):
    gen = _gen(M + N + K)
    A = torch.randn((M, K), generator=gen).to(TYPES[dtype]).cuda()
    W = lc.random_w4(gen, (), N, K, group, asym, A.dtype)
    D = torch.full((M, N), float("nan"), dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=A.device)
    lc.check(D, *_product_ref(A, W), f"{M}x{N}x{K} group {group}")


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (5, 16384, 1024), (64, 1024, 16384), (1, 8, 65536), (3, 40000, 256),
                                   (200, 8192, 1024)])
def test_long_products(M, N, K):
    gen = _gen(M + N)
    A = torch.randn((M, K), generator=gen).bfloat16().cuda()
    W = lc.random_w4(gen, (), N, K, 128, False, A.dtype)
    D = torch.full((M, N), float("nan"), dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    g.gemm_f16_nt_check(device=A.device)
    lc.check(D, *_product_ref(A, W), f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 6, 40, 64, 100])
def test_product_with_epilogue(dtype, M):
    N, K = 136, 352
    gen = _gen(M)
    A = torch.randn((M, K), generator=gen).to(TYPES[dtype]).cuda()
    W = lc.random_w4(gen, (), N, K, 32, True, A.dtype)
    C = torch.randn((M, N), generator=gen).to(A.dtype).cuda()
    bias = torch.randn(N, generator=gen).to(A.dtype).cuda()
    s = (torch.rand(N, generator=gen) + 0.5).cuda()
    ref, tol = _product_ref(A, W)
    lin = 1.5 * s.double() * ref
    full = lin - 0.5 * C.double() + bias.double()
    ltol = 1.5 * s.double() * (tol - 1.01 * lc.U[A.dtype] * ref.abs()) + 1.01 * lc.U[A.dtype] * full.abs() \
        + 2.0 ** -21 * (lin.abs() + C.double().abs() + bias.double().abs()) + lc.FLOOR
    D = C.clone()                                   # in place: C is D
    g.gemm_w4_nt(A, W, D, alpha=1.5, beta=-0.5, C=D, bias=bias, scale_n=s, activation=g.Activation.RELU)
    g.gemm_f16_nt_check(device=A.device)
    lc.check(D, full.clamp(min=0), ltol, "epilogue")
    # K = 0: the empty sum
    D0 = torch.full((M, N), float("nan"), dtype=A.dtype, device="cuda")
    W0 = g.W4(torch.empty((N, 0), dtype=torch.uint8, device="cuda"), torch.empty((0, N), dtype=A.dtype, device="cuda"),
              None, 32)
    g.gemm_w4_nt(A[:, :0].contiguous(), W0, D0, bias=bias)
    assert torch.equal(D0, bias.expand(M, N))
    g.gemm_w4_nt(A[:0], W, D0[:0])


@pytest.mark.parametrize("M", [3, 20, 64, 70])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(M):
    N, K = 264, 1056
    gen = _gen(M)
    A = torch.randn((M, K), generator=gen).half().cuda()
    W = lc.random_w4(gen, (), N, K, 32, True, A.dtype)
    ref, tol = _product_ref(A, W)
    A[1, 17], A[2, K - 1] = float("inf"), float("nan")
    W.scales[5, 9] = float("nan")
    D = torch.zeros((M, N), dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, D)
    fine = torch.ones((M, N), dtype=torch.bool, device="cuda")
    fine[1:3] = False
    fine[:, 9] = False
    assert not bool(torch.isfinite(D[1:3]).any()) and not bool(torch.isfinite(D[:, 9]).any())
    lc.check(D[fine], ref[fine], tol[fine], "other rows and columns")


def test_product_writes_only_its_output_and_twice_the_same():
    M, N, K = 13, 1000, 1024
    gen = _gen(1)
    A = torch.randn((M, K), generator=gen).half().cuda()
    W = lc.random_w4(gen, (), N, K, 64, True, A.dtype)
    room = torch.full((M + 2, N), 7.0, dtype=A.dtype, device="cuda")
    g.gemm_w4_nt(A, W, room[1:M + 1])
    first = room.clone()
    g.gemm_w4_nt(A, W, room[1:M + 1])
    assert torch.equal(first, room)
    assert bool((room[0] == 7).all()) and bool((room[M + 1] == 7).all())


@pytest.mark.parametrize("M", [4, 100])
def test_other_stream_and_graph(M):
    N, K = 520, 768
    gen = _gen(2)
    W = lc.random_w4(gen, (), N, K, 128, False, torch.bfloat16)
    A = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        A.copy_(torch.randn((M, K), generator=gen))
        g.gemm_w4_nt(A, W, D)
        rows = torch.randn((16, K), generator=gen).bfloat16().cuda()
        packed = g.gemm_w4_quantize(rows, 32)
    s.synchronize()
    lc.check(D, *_product_ref(A, W), "other stream")
    assert torch.equal(packed.codes, lc.quantize64(rows, 32, False)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.gemm_w4_nt(A, W, D, stream=s)
    for _ in range(3):
        A.copy_(torch.randn((M, K), generator=gen))
        D.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        lc.check(D, *_product_ref(A, W), "replay")


def test_codes_past_two_to_the_31():
    # a stack of 2^32 + weights: offsets of codes and values pass 32 bits
    B, N, K = 5, 8192, 131072
    W = torch.zeros((B, N, K), dtype=torch.float16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    W[-1, -64:].normal_(generator=gen)
    out = g.gemm_w4_quantize(W, 128)
    tail = W[-1, -64:].contiguous()
    codes, scales, _ = lc.quantize64(tail, 128, False)
    assert torch.equal(out.codes[-1, -64:], codes) and torch.equal(out.scales[-1, :, -64:], scales)
    assert bool((out.codes[0, :8] == 0x88).all())
    del W
    values = g.gemm_w4_dequantize(out)
    one = g.W4(codes, scales.contiguous(), None, 128)
    assert torch.equal(values[-1, -64:], lc.w64(one)[0].float().half())


def test_refusals():
    A = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    W = lc.random_w4(_gen(0), (), 16, 64, 32, True, torch.float16)
    D = torch.zeros((4, 16), dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        g.gemm_w4_nt(A.float(), W, D)
    with pytest.raises(TypeError):
        g.gemm_w4_nt(A.bfloat16(), W, D)
    with pytest.raises(TypeError):
        g.gemm_w4_nt(A, W.codes, D)
    with pytest.raises(ValueError):
        g.gemm_w4_nt(A, W, D.t().contiguous())
    with pytest.raises(ValueError):
        g.gemm_w4_nt(A, W, torch.zeros((16, 4), dtype=torch.float16, device="cuda").t())
    with pytest.raises(ValueError):
        g.gemm_w4_nt(A.cpu(), W, D)
    with pytest.raises(ValueError):
        g.gemm_w4_nt(A, g.W4(W.codes, W.scales, W.zeros, 16), D)
    with pytest.raises(ValueError):
        g.gemm_w4_nt(A, g.W4(W.codes, W.scales[:1], W.zeros, 32), D)
    with pytest.raises(ValueError):
        g.gemm_w4_quantize(A, 128)
    with pytest.raises(ValueError):
        g.gemm_w4_quantize(A, 32, zeros=W.zeros, symmetric=True)
    with pytest.raises(g.GemmError) as e:        # 12 rows: a row of scales is not whole 16-byte units
        g.gemm_w4_quantize(torch.zeros((12, 64), dtype=torch.float16, device="cuda"), 32)
    assert e.value.status == g.Status.ERR_MISALIGNED
    shifted = torch.zeros(4 * 64 + 4, dtype=torch.float16, device="cuda")[4:].view(4, 64)   # 8 bytes off
    with pytest.raises(g.GemmError) as e:
        g.gemm_w4_nt(shifted, W, D)
    assert e.value.status == g.Status.ERR_MISALIGNED
    with pytest.raises(g.GemmError) as e:
        g.gemm_w4_nt(A, W, A.view(-1)[:64].view(4, 16))
    assert e.value.status == g.Status.ERR_INVALID_VALUE
