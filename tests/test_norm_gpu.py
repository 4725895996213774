"""RMS norm with the residual's addition and an 8-bit output, against 64 bits.

Bounds, fixed from the arithmetic before any run.  The sum of squares takes at
most n = 8 ceil(H / 8192) additions in one thread (32 up to 32768 columns) and ten
between threads, all of positive numbers, each off by at most 2^-24 of the sum;
the root halves that; the sum x + r, the division by H, the addition of eps, the root and the two products of y are one
rounding each.  So y is off by at most (n + 10) / 2 + 6 roundings of 2^-24, and the
scale by one more (the quotient).
"""
import math

import pytest
import torch

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half a step relative to the value, half the spacing of subnormal numbers, largest
U8 = {torch.float8_e4m3fn: (2.0 ** -4, 2.0 ** -10, 448.0), torch.float8_e5m2: (2.0 ** -3, 2.0 ** -17, 57344.0)}


def draw(T, H, dtype, seed, residual=True, weight=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=gen, device=DEV)
    x *= torch.exp2(torch.randint(-3, 4, (T, 1), generator=gen, device=DEV).float())
    r = torch.randn(T, H, generator=gen, device=DEV).to(dtype) if residual else None
    w = (torch.randn(H, generator=gen, device=DEV) * 0.5 + 1.0).to(dtype) if weight else None
    return x.to(dtype), r, w


def roundings(H):
    return (max(32, 8 * math.ceil(H / 8192)) + 10) / 2 + 6


def check(out, x, r, w, eps, H, total=None):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * (1.0 if w is None else w.double())
    off = roundings(H) * 2.0 ** -24
    if total is not None:
        assert bool(((total.double() - h).abs() <= 1.01 * U[x.dtype] * h.abs() + 2.0 ** -25).all())
    if out.Y is not None:
        assert bool(((out.Y.double() - y).abs() <= (1.01 * U[x.dtype] + off) * y.abs() + 2.0 ** -25).all())
    if out.Y8 is not None:
        u, floor, top = U8[out.Y8.dtype]
        if out.scales is not None:
            want = y.abs().amax(1) / top
            assert bool(((out.scales.double() - want).abs() <= (off + 2.0 ** -24) * want).all())
            s = out.scales.double()[:, None]
        else:
            s = check.scale
        t = torch.where(y == 0, 0.0, y / s)
        q = out.Y8.to(torch.float32).double()
        bad = ~((q - t.clamp(-top, top)).abs() <= (u + off + 2.0 ** -23) * t.abs().clamp(max=top) + floor)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())
    return y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (1, 2048), (5, 248), (37, 5128), (2, 8192), (2, 8200), (1, 16384),
                                 (3, 16392), (2, 32768), (2, 32776), (1, 100000), (305, 256), (306, 1024), (1000, 1032),
                                 (700, 4096), (400, 8192), (310, 11000), (306, 20000), (4096, 24)])
def test_all_outputs(T, H, dtype):
    x, r, w = draw(T, H, dtype, T + H)
    for kind in (torch.float8_e4m3fn, torch.float8_e5m2):
        total, Y = torch.empty_like(x), torch.empty_like(x)
        out = g.gemm_rmsnorm(x, w, r, 1e-5, Y=Y, Y8=torch.empty(T, H, dtype=kind, device=DEV), total=total)
        assert out.Y is Y and out.total is total
        check(out, x, r, w, 1e-5, H, total)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("H", [72, 4096, 40000])
def test_parts_left_out(residual, weight, H):
    x, r, w = draw(9, H, torch.bfloat16, H, residual, weight)
    check(g.gemm_rmsnorm(x, w, r), x, r, w, 1e-6, H)
    out = g.gemm_rmsnorm(x, w, r, Y8=g.Dtype.E4M3)
    assert out.Y is None and out.total is None and out.Y8.dtype == torch.float8_e4m3fn
    check(out, x, r, w, 1e-6, H)
    check.scale = 0.011
    out = g.gemm_rmsnorm(x, w, r, Y8=g.Dtype.E5M2, scale=check.scale)
    assert out.scales is None
    check(out, x, r, w, 1e-6, H)


@pytest.mark.parametrize("scale", [2.0 ** -9, 0.02])
def test_given_scale_saturates(scale):
    x, r, w = draw(20, 512, torch.float16, 3)
    check.scale = scale
    check(g.gemm_rmsnorm(x, w, r, Y8=g.Dtype.E4M3, scale=scale), x, r, w, 1e-6, 512)


@pytest.mark.parametrize("T,H", [(3, 640), (400, 8192), (2, 40000), (2000, 4104), (20001, 72), (700, 16384), (2000, 11000)])
def test_in_place(T, H):
    """total over the residual and Y over X, or the other way round, change nothing."""
    x, r, w = draw(T, H, torch.bfloat16, 11)
    total = torch.empty_like(x)
    want = g.gemm_rmsnorm(x, w, r, total=total, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        out = g.gemm_rmsnorm(a, w, b, total=a if swap else b, Y=b if swap else a, Y8=g.Dtype.E4M3)
        for got, ref in zip((out.Y, out.total, out.scales), (want.Y, total, want.scales)):
            assert torch.equal(got, ref)
        assert torch.equal(out.Y8.view(torch.uint8), want.Y8.view(torch.uint8))


def test_zero_rows_and_special_values():
    x, r, w = draw(6, 1024, torch.bfloat16, 5)
    x[1], r[1] = 0, 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] *= 2.0 ** -60       # mean square far below eps
    r[4] *= 2.0 ** -60
    out = g.gemm_rmsnorm(x, w, r, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
    assert float(out.scales[1]) == 0 and int(out.Y8.view(torch.uint8)[1].sum()) == 0 and not bool(out.Y[1].any())
    assert bool(out.Y[2].isnan().all()) and bool(out.Y8[2].float().isnan().all()) and bool(out.scales[2].isnan())
    assert bool(out.Y[3, 9].isnan()) and not bool(out.Y[3, :9].any()) and bool(out.scales[3].isnan())
    keep = torch.tensor([0, 4, 5], device=DEV)
    check(g.llm.Normed(out.Y[keep], out.Y8[keep], out.scales[keep], None), x[keep], r[keep], w, 1e-6, 1024)


def test_tiny_weights_and_no_eps():
    """Scales near fp32's smallest numbers: codes still use the whole range."""
    x, _, _ = draw(4, 512, torch.bfloat16, 6, residual=False, weight=False)
    w = torch.full((512,), 2.0 ** -120, device=DEV, dtype=torch.bfloat16)
    out = g.gemm_rmsnorm(x, w, eps=0.0, Y8=g.Dtype.E4M3)
    # the scale is a subnormal number of 2^-149 steps: about 2^-126.5, off by up to 2^-150
    y = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True)) * 2.0 ** -120
    want = y.abs().amax(1) / 448
    assert bool(((out.scales.double() - want).abs() <= 2.0 ** -149 + 2.0 ** -20 * want).all())
    t = (y / out.scales.double()[:, None]).clamp(-448, 448)
    assert bool(((out.Y8.float().double() - t).abs() <= (2.0 ** -4 + 2.0 ** -18) * t.abs() + 2.0 ** -10).all())


def test_same_result_again():
    x, r, w = draw(320, 1024, torch.bfloat16, 8)
    many = g.gemm_rmsnorm(x, w, r, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
    again = g.gemm_rmsnorm(x, w, r, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
    assert torch.equal(many.Y, again.Y) and torch.equal(many.scales, again.scales)
    check(many, x, r, w, 1e-6, 1024)


def test_nothing_is_written_beyond_the_rows():
    T, H = 3, 200
    x, r, w = draw(T, H, torch.float16, 9)
    for kind in (torch.float16, torch.float8_e4m3fn):
        wide = torch.full((T + 2, H), 7.0, device=DEV).to(kind)
        part = wide[1:T + 1] if kind == torch.float8_e4m3fn and H % 16 == 0 else wide.view(-1)[: T * H].view(T, H)
        g.gemm_rmsnorm(x, w, r, **({"Y": part} if kind == torch.float16 else {"Y8": part}))
        assert bool((wide.view(-1)[T * H:].float() == 7.0).all())


def test_graph_streams_and_empty():
    x, r, w = draw(40, 2048, torch.bfloat16, 10)
    want = g.gemm_rmsnorm(x, w, r, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y, Y8, sc = torch.zeros_like(x), torch.empty_like(want.Y8), torch.zeros_like(want.scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.gemm_rmsnorm(x, w, r, Y=Y, Y8=Y8, scales=sc)
    x.mul_(2.0), r.mul_(2.0)     # y stays but for eps
    graph.replay()
    torch.cuda.synchronize()
    check(g.llm.Normed(Y, Y8, sc, None), x, r, w, 1e-6, 2048)
    e = g.gemm_rmsnorm(x[:0], w, r[:0], Y8=g.Dtype.E4M3)
    assert e.Y8.shape == (0, 2048)
    g.gemm_f16_nt_check(device=DEV)


def test_refusals():
    x, r, w = draw(4, 64, torch.float16, 1)
    bad = [
        (TypeError, dict(X=x.float())), (TypeError, dict(weight=w.bfloat16())), (ValueError, dict(weight=w[:32])),
        (ValueError, dict(residual=r[:2])), (ValueError, dict(X=x.t())), (ValueError, dict(scales=torch.empty(4, device=DEV))),
        (ValueError, dict(scale=0.5)), (ValueError, dict(Y8=g.Dtype.E4M3, scale=-1.0)), (ValueError, dict(Y8=g.Dtype.E4M3, scale=float("nan"))),
        (TypeError, dict(Y8=g.Dtype.F16)), (TypeError, dict(Y8=torch.empty_like(x))), (ValueError, dict(X=x.cpu())),
        (ValueError, dict(Y8=g.Dtype.E4M3, scales=torch.empty(3, device=DEV))), (g.GemmError, dict(eps=-1.0)),
        (g.GemmError, dict(eps=float("inf"))), (g.GemmError, dict(Y=x, total=x)), (ValueError, dict(X=x[0])),
    ]
    for error, change in bad:
        args = dict(X=x, weight=w, residual=r) | change
        with pytest.raises(error):
            g.gemm_rmsnorm(**args)
    with pytest.raises(g.GemmError):
        g.gemm_rmsnorm(torch.empty(4, 60, dtype=torch.float16, device=DEV))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(3, 512), (2, 40000), (700, 8192)])
def test_given_scales_of_any_size(T, H, dtype):
    """A quotient y / scale beyond fp32's numbers gives the largest code, not NaN: scales down to fp32's smallest
    number, which is not a normal one."""
    x, r, w = draw(T, H, dtype, 4)
    for kind in (g.Dtype.E4M3, g.Dtype.E5M2):
        for scale in (2.0 ** -149, 1e-38, 2.0 ** -101, 2.0 ** -99, 1e-30, 1e5, 3e38):
            check.scale = float(torch.tensor(scale))
            out = g.gemm_rmsnorm(x, w, r, Y8=kind, scale=scale)
            assert not bool(out.Y8.float().isnan().any())
            check(out, x, r, w, 1e-6, H)


def test_given_scale_below_large_rows():
    """y near fp32's largest number over a scale of ordinary size."""
    x, r, _ = draw(5, 1024, torch.bfloat16, 14)
    w = torch.full((1024,), 2.0 ** 124, device=DEV, dtype=torch.bfloat16)
    for scale in (0.0078125, 2.0 ** -110):
        check.scale = scale
        check(g.gemm_rmsnorm(x, w, r, Y8=g.Dtype.E4M3, scale=scale), x, r, w, 1e-6, 1024)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(39001, 24), (39001, 64), (40000, 96), (1300, 4096), (700, 8192), (500, 11000), (400, 16384)])
def test_rows_of_ctas_that_stay(T, H, dtype):
    """Enough rows that CTAs take several, with one to four pieces per thread, in every output."""
    x, r, w = draw(T, H, dtype, T + H)
    total, Y = torch.empty_like(x), torch.empty_like(x)
    check(g.gemm_rmsnorm(x, w, r, 1e-5, Y=Y, Y8=g.Dtype.E4M3, total=total), x, r, w, 1e-5, H, total)
    check(g.gemm_rmsnorm(x, w), x, None, w, 1e-6, H)
    check(g.gemm_rmsnorm(x, Y8=g.Dtype.E5M2), x, None, None, 1e-6, H)


@pytest.mark.parametrize("T,H", [(3, 208), (700, 8192), (2, 40000)])
def test_nothing_is_written_around_the_rows(T, H):
    x, r, w = draw(T, H, torch.float16, 9)
    wide = [torch.full((T + 2, H), 7.0, device=DEV).to(kind) for kind in (x.dtype, torch.float8_e4m3fn, x.dtype)]
    scales = torch.full((T + 2,), 7.0, device=DEV)
    Y, Y8, total = (t[1:T + 1] for t in wide)
    check(g.gemm_rmsnorm(x, w, r, Y=Y, Y8=Y8, scales=scales[1:T + 1], total=total), x, r, w, 1e-6, H, total)
    for t in (*wide, scales):
        assert bool((t[0].float() == 7.0).all()) and bool((t[T + 1].float() == 7.0).all())


def test_products_with_the_weight_below_normal_numbers():
    """The scale has the bits that max|h w| has in fp32, half a step of 2^-149; Y keeps all of its own."""
    for h, w in ((2.0 ** -60, 2.0 ** -80), (2.0 ** -62, 2.0 ** -86), (2.0 ** -60, 2.0 ** -95)):
        x = draw(4, 512, torch.bfloat16, 6, residual=False, weight=False)[0] * h
        W = torch.full((512,), w, device=DEV, dtype=torch.bfloat16)
        out = g.gemm_rmsnorm(x, W, eps=0.0, Y=torch.empty_like(x), Y8=g.Dtype.E4M3)
        v = x.double()
        root = 1 / torch.sqrt((v * v).mean(1))
        y, top = v * root[:, None] * w, v.abs().amax(1) * w
        off = roundings(512) * 2.0 ** -24
        assert bool(((out.Y.double() - y).abs() <= (1.01 * U[x.dtype] + off) * y.abs()).all())
        assert bool(((out.scales.double() - top * root / 448).abs() <= 1.01 * 2.0 ** -150 * root / 448 + 2 * off * top * root / 448).all())
        if w == 2.0 ** -95:
            assert not bool(out.scales.any()) and not bool(out.Y8.float().any())
