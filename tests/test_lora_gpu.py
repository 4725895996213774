"""Low-rank adapters of many requests beside a projection, against 64 bits.

Bounds per element, fixed from the arithmetic before any run; u is half a unit in the
last place (2^-11 for fp16, 2^-8 for bf16), taken 1 % wider:
  V = X Aᵀ in fp32: a chain of at most K / 128 MMAs in a warp, 8 warps and at most 32
      pieces are added, each addition off by at most 2^-23 of the magnitudes that enter
  V cut into hi + lo: off by 2^-17 of it (bf16; fp16 less), or 2^-24 of the row's largest
      where fp16 runs out of small numbers
  times B: R / 8 MMAs (hi and lo), the factor, beta C: 2^-23 each
  one rounding of U: u |U|;  D: u |D| and 2^-22 of the projection's magnitudes besides
"""
import pytest
import torch

import dense_fp16_gemm_f16_gb300 as g
from llm_check import E32, FLOOR, U as UNIT, random_w4, w64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]


def draw(M, N, K, R, count, dtype, seed, runs=False, none=0.15):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return (torch.randn(*shape, generator=gen, device=DEV) * shape[-1] ** -0.5).to(dtype)

    X = torch.randn(M, K, generator=gen, device=DEV).to(dtype)
    lora = g.Lora(normal(count, R, K), normal(count, N, R), torch.rand(count, generator=gen, device=DEV) + 0.25)
    ids = torch.randint(0, max(count, 1), (M,), generator=gen, device=DEV, dtype=torch.int32)
    if runs:
        ids = ids.sort().values
    ids[torch.rand(M, generator=gen, device=DEV) < none] = -1
    return X, lora, ids, gen


def delta64(X, lora, ids, beta=0.0, C=None):
    """(beta C + the adapters' part, the error that may come before its rounding)."""
    M, K = X.shape
    count, R, _ = lora.A.shape
    ref = torch.zeros(M, lora.B.shape[1], dtype=torch.float64, device=X.device)
    err = torch.zeros_like(ref)
    for a in range(count):
        rows = (ids == a).nonzero(as_tuple=True)[0]
        if not len(rows):
            continue
        x, A, B = X[rows].double(), lora.A[a].double(), lora.B[a].double()
        f = 1.0 if lora.factors is None else lora.factors[a].double()
        V, mag = x @ A.T, x.abs() @ A.abs().T
        ref[rows] = f * (V @ B.T)
        eV = (K / 128 + 44) * 2.0 ** -23 * mag + 2.0 ** -17 * V.abs() + 2.0 ** -24 * V.abs().amax(1, keepdim=True)
        err[rows] = abs(f) * ((eV + (R / 8 + 4) * 2.0 ** -23 * V.abs()) @ B.abs().T)
    if C is not None:
        ref += beta * C.double()
        err += 2.0 ** -22 * abs(beta) * C.double().abs()
    return ref, err


def check(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} out of bounds, worst "
                                 f"{float(((got.double() - ref).abs() / tol)[bad].max())}, first at {bad.nonzero()[0].tolist()}")


SIZES = [  # M, N, K, R, count
    (1, 8, 8, 8, 1), (1, 1024, 2048, 8, 4), (3, 40, 72, 16, 2), (16, 8192, 1024, 16, 32), (17, 264, 520, 24, 3),
    (33, 1000, 4104, 40, 40), (64, 2048, 1032, 64, 5), (61, 512, 8192, 128, 48), (9, 320, 256, 256, 4), (130, 600, 264, 136, 7),
    (200, 72, 2048, 32, 1), (255, 136, 512, 8, 300), (256, 1032, 520, 16, 64), (257, 512, 512, 16, 3), (400, 328, 1000, 72, 500),
    (1000, 2048, 1024, 64, 8), (2048, 520, 2056, 16, 1), (8200, 64, 256, 24, 40), (9500, 136, 4096, 16, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,R,count", SIZES)
def test_delta(M, N, K, R, count, dtype):
    for runs in (False, True):
        X, lora, ids, gen = draw(M, N, K, R, count, dtype, M + N + R, runs)
        ref, err = delta64(X, lora, ids)
        U = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
        assert g.gemm_lora_delta(X, lora, ids, U) is U
        check(U, ref, 1.01 * UNIT[dtype] * ref.abs() + err + FLOOR)
        C = torch.randn(M, N, generator=gen, device=DEV).to(dtype)
        ref, err = delta64(X, lora, ids, -0.7, C)
        assert g.gemm_lora_delta(X, lora, ids, U, beta=-0.7, C=C) is U
        check(U, ref, 1.01 * UNIT[dtype] * ref.abs() + err + FLOOR)
        E = C.clone()
        g.gemm_lora_delta(X, lora, ids, E, beta=-0.7, C=E)
        assert torch.equal(E, U)
    g.gemm_f16_nt_check(device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,R,count", [(1, 1024, 2048, 8, 4), (1, 40, 4096, 256, 2), (4, 136, 512, 256, 3), (16, 8192, 1024, 16, 32), (17, 264, 520, 24, 3),
                                           (33, 8192, 520, 24, 9), (64, 1000, 8192, 16, 70), (60, 12000, 264, 8, 5), (64, 2048, 1032, 64, 5),
                                           (65, 72, 136, 16, 2), (250, 5000, 1032, 32, 64), (256, 256, 8192, 16, 9),
                                           (512, 2048, 4096, 128, 8), (3000, 4104, 1024, 16, 4), (8300, 520, 512, 8, 3)])
def test_projection_with_adapters(M, N, K, R, count, dtype):
    X, lora, ids, gen = draw(M, N, K, R, count, dtype, M + K, runs=M > 256)
    W = (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).to(dtype)
    C, bias = (torch.randn(s, generator=gen, device=DEV).to(dtype) for s in ((M, N), (N,)))
    sn = torch.rand(N, generator=gen, device=DEV) + 0.5
    for args in (dict(), dict(alpha=0.6, beta=1.0, C=C, bias=bias, scale_n=sn, activation=g.Activation.RELU)):
        D = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
        g.gemm_lora_nt(X, W, lora, ids, D, **args)
        part, err = delta64(X, lora, ids, args.get("beta", 0.0), args.get("C"))
        f = (args.get("alpha", 1.0) * (sn.double() if args else 1.0))
        x, w = X.double(), W.double()
        ref, mag = (x @ w.T) * f + part, (x.abs() @ w.abs().T) * f
        if args:
            ref = ref + bias.double()
        tol = UNIT[dtype] * 1.01 * (ref.abs() + part.abs()) + err + E32 * (mag + part.abs() + 4) + 2 * FLOOR
        check(D, ref.clamp(min=0) if args else ref, tol)
        if M > 16 or M * R > 1024:   # the same as the two calls that it then stands for
            T, E = (torch.empty_like(D) for _ in range(2))
            g.gemm_lora_delta(X, lora, ids, T, beta=args.get("beta", 0.0), C=args.get("C"))
            g.gemm_nt_ex(X, W, E, **(args | dict(beta=1.0, C=T)))
            assert torch.equal(D, E)
        if "C" in args:
            E = C.clone()
            g.gemm_lora_nt(X, W, lora, ids, E, **(args | dict(C=E)))
            assert torch.equal(D, E)
    # rows without an adapter, and all rows with none: the plain product
    D, P = (torch.empty(M, N, dtype=dtype, device=DEV) for _ in range(2))
    g.gemm_lora_nt(X, W, lora, ids, D)
    g.gemm_nt_ex(X, W, P)
    assert torch.equal(D[ids < 0], P[ids < 0])
    g.gemm_lora_nt(X, W, lora, torch.full_like(ids, count), D)
    assert torch.equal(D, P)
    g.gemm_f16_nt_check(device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,group,asym", [(1, 128, False), (13, 32, True), (40, 64, False), (64, 128, True), (300, 64, True)])
def test_beside_4_bit_weights(M, group, asym, dtype):
    N, K = 1032, 1024
    X, lora, ids, gen = draw(M, N, K, 16, 6, dtype, M)
    W = random_w4(torch.Generator().manual_seed(M), (), N, K, group, asym, dtype, DEV)
    C, bias = (torch.randn(s, generator=gen, device=DEV).to(dtype) for s in ((M, N), (N,)))
    D, E = (torch.empty(M, N, dtype=dtype, device=DEV) for _ in range(2))
    g.gemm_lora_nt(X, W, lora, ids, D, beta=0.5, C=C, bias=bias)
    g.gemm_w4_nt(X, W, E, beta=1.0, C=g.gemm_lora_delta(X, lora, ids, beta=0.5, C=C), bias=bias)
    assert torch.equal(D, E)
    if M <= 16:
        w, wm = w64(W)
        part, err = delta64(X, lora, ids, 0.5, C)
        ref = X.double() @ w.T + part + bias.double()
        tol = UNIT[dtype] * 1.01 * (ref.abs() + part.abs()) + err + E32 * (X.double().abs() @ wm.T + part.abs() + 8) + 2 * FLOOR
        check(D, ref, tol)


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("M", [1, 30, 64, 300])
def test_norm_adapters_and_8_bit_product(M, kind):
    """A step of a decoder: norm of the summed stream, its 16-bit rows to the adapters, its 8-bit rows to the
    projection, all in one graph that is replayed on other activations."""
    N, K, dtype = 1024, 2048, torch.bfloat16
    X, lora, ids, gen = draw(M, N, K, 16, 5, dtype, M)
    r, w = torch.randn(M, K, generator=gen, device=DEV).to(dtype), (torch.rand(K, generator=gen, device=DEV) + 0.5).to(dtype)
    top = 448.0 if kind == torch.float8_e4m3fn else 57344.0
    W = (torch.randn(N, K, generator=gen, device=DEV) * top / 5).clamp(-top, top).to(kind)
    sn = (torch.rand(N, generator=gen, device=DEV) + 0.5) * K ** -0.5 * 5 / top
    Y, Y8, total = torch.empty_like(X), torch.empty(M, K, dtype=kind, device=DEV), torch.empty_like(X)
    scales, T, D = torch.empty(M, device=DEV), torch.empty(M, N, dtype=dtype, device=DEV), torch.empty(M, N, dtype=dtype, device=DEV)

    def step():
        g.gemm_rmsnorm(X, w, r, Y=Y, Y8=Y8, scales=scales, total=total)
        g.gemm_lora_delta(Y, lora, ids, T)
        g.gemm_nt_ex(Y8, W, D, scale_m=scales, scale_n=sn, beta=1.0, C=T)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for i in range(4):
            X.copy_(torch.randn(X.shape, generator=gen, device=DEV))
            ids.copy_(torch.randint(-1, 5, ids.shape, generator=gen, device=DEV))
            graph.replay()
    torch.cuda.synchronize()
    part, err = delta64(Y, lora, ids)
    check(T, part, 1.01 * UNIT[dtype] * part.abs() + err + FLOOR)
    a, b = Y8.float().double() * scales.double()[:, None], W.float().double() * sn.double()[:, None]
    ref = a @ b.T + T.double()
    check(D, ref, 1.01 * UNIT[dtype] * ref.abs() + (K / 32 + 6) * 2.0 ** -23 * (a.abs() @ b.abs().T + T.double().abs()))
    assert torch.equal(total, (X.float() + r.float()).to(dtype))
    g.gemm_f16_nt_check(device=DEV)


def test_special_values_stay_in_their_rows_and_adapters():
    M, N, K, R = 40, 264, 512, 16
    X, lora, ids, _ = draw(M, N, K, R, 4, torch.float16, 3, none=0.0)
    ids = torch.arange(M, device=DEV, dtype=torch.int32) % 4
    want = g.gemm_lora_delta(X, lora, ids)
    X[5, 3], X[6, 4] = float("nan"), float("inf")
    lora.A[1, 0, 0] = float("nan")      # adapter 1 is not to be used
    lora.B[1] = float("inf")
    ids[ids == 1] = 7
    ids[0], ids[2] = -2 ** 31, 2 ** 31 - 1
    got = g.gemm_lora_delta(X, lora, ids)
    none = (ids < 0) | (ids >= 4)
    assert int(none.sum()) >= 12 and not bool(got[none].any())
    keep = ~none
    keep[5], keep[6] = False, False
    assert torch.equal(got[keep], want[keep])
    if not bool(none[5]):
        assert bool(got[5].isnan().all())
    assert not bool(got[6].isfinite().any())


@pytest.mark.parametrize("M", [12, 40])
def test_special_values_beside_a_projection(M):
    """Adapters that no row uses are not read; an infinity or NaN in a row of X stays in that row."""
    N, K, R = 264, 512, 16
    X, lora, ids, gen = draw(M, N, K, R, 4, torch.bfloat16, 13)
    W = (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).bfloat16()
    ids[ids == 2] = -7
    D, E = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gemm_lora_nt(X, W, lora, ids, D)
    lora.A[2], lora.B[2], lora.factors[2] = float("nan"), float("inf"), float("nan")
    X[1, 5], X[3, 7] = float("nan"), float("-inf")
    g.gemm_lora_nt(X, W, lora, ids, E)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[1], keep[3] = False, False
    assert torch.equal(D[keep], E[keep])
    assert bool(E[1].isnan().all()) and not bool(E[3].isfinite().any())


@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_small_inner_values(dtype):
    """X Aᵀ may lie far outside fp16's range: only U is a number of the type."""
    M, N, K, R = 20, 128, 1024, 16
    X, lora, ids, _ = draw(M, N, K, R, 3, dtype, 8)
    big, small = 2.0 ** 12, 2.0 ** -12
    up = g.Lora(lora.A * big, lora.B * small, lora.factors)
    X2 = X * big
    ref, err = delta64(X2, up, ids)
    check(g.gemm_lora_delta(X2, up, ids) , ref, 1.01 * UNIT[dtype] * ref.abs() + err + FLOOR)
    down = g.Lora((lora.A * small).to(dtype), lora.B, torch.full((3,), 2.0 ** 14, device=DEV))
    ref, err = delta64(X, down, ids)
    check(g.gemm_lora_delta(X, down, ids), ref, 1.01 * UNIT[dtype] * ref.abs() + err + FLOOR)


def test_a_row_does_not_depend_on_its_place():
    """Rows in another order give the same rows: sums do not depend on what shares a tile."""
    M, N, K = 200, 520, 1024
    X, lora, ids, gen = draw(M, N, K, 32, 9, torch.bfloat16, 4)
    want = g.gemm_lora_delta(X, lora, ids)
    p = torch.randperm(M, generator=gen, device=DEV)
    assert torch.equal(g.gemm_lora_delta(X[p], lora, ids[p]), want[p])
    assert torch.equal(g.gemm_lora_delta(X, lora, ids), want)


@pytest.mark.parametrize("M,R", [(16, 32), (300, 16), (5000, 40)])
def test_same_result_again(M, R):
    """Which rows share a unit of work may change from run to run; results do not."""
    X, lora, ids, _ = draw(M, 520, 1032, R, 7, torch.float16, M)
    want = g.gemm_lora_delta(X, lora, ids)
    for _ in range(10):
        assert torch.equal(g.gemm_lora_delta(X, lora, ids), want)


def test_two_host_threads_on_one_stream():
    """Calls of two threads on one stream share its scratch and keep out of each other's way."""
    import threading
    N, K = 264, 520
    stream = torch.cuda.Stream()
    jobs = []
    for i, M in enumerate((10, 400)):
        X, lora, ids, gen = draw(M, N, K, 16, 5, torch.bfloat16, i)
        W = (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).bfloat16()
        D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        g.gemm_lora_nt(X, W, lora, ids, D, stream=stream)
        stream.synchronize()
        jobs.append((X, W, lora, ids, D, D.clone()))
    failed = []

    def work(job):
        X, W, lora, ids, D, want = job
        for _ in range(40):
            g.gemm_lora_nt(X, W, lora, ids, D, stream=stream)
            stream.synchronize()
            if not torch.equal(D, want):
                failed.append(len(X))

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    g.gemm_f16_nt_check(device=DEV)


def test_a_part_of_a_batch():
    """Slices of a batch, whose ids begin anywhere, give the batch's rows."""
    X, lora, ids, _ = draw(90, 264, 520, 16, 5, torch.bfloat16, 12)
    ref, err = delta64(X, lora, ids)
    for first, last in ((1, 12), (5, 90), (3, 40)):
        got = g.gemm_lora_delta(X[first:last], lora, ids[first:last])
        r = ref[first:last]
        check(got, r, 1.01 * UNIT[torch.bfloat16] * r.abs() + err[first:last] + FLOOR)
        W = torch.zeros(264, 520, dtype=torch.bfloat16, device=DEV)
        D = torch.empty_like(got)
        g.gemm_lora_nt(X[first:last], W, lora, ids[first:last], D)
        check(D, r, 2.02 * UNIT[torch.bfloat16] * r.abs() + 2 * err[first:last] + FLOOR)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,H,I,R", [(1, 2048, 1024, 16), (7, 1024, 520, 64), (16, 8192, 1032, 24), (40, 1024, 2048, 16),
                                     (300, 1024, 520, 32)])
def test_layers_without_a_pause(M, H, I, R, dtype):
    """Norms and products that start while the one before them drains, over the same few buffers: the same as with
    a synchronisation after every call, and in a graph."""
    X, up, ids, gen = draw(M, I, H, R, 5, dtype, M + H)
    _, down, _, _ = draw(1, H, I, R, 5, dtype, M + I)
    W1, W2 = ((torch.randn(s, generator=gen, device=DEV) * s[1] ** -0.5).to(dtype) for s in ((I, H), (H, I)))
    w = (torch.rand(H, generator=gen, device=DEV) + 0.5).to(dtype)
    x, y, h = torch.empty_like(X), torch.empty_like(X), torch.empty(M, I, dtype=dtype, device=DEV)

    def layers(between):
        x.copy_(X)
        for i in range(6):
            g.gemm_rmsnorm(x, w, Y=y)
            between()
            g.gemm_lora_nt(y, W1, up, ids, h, activation=g.Activation.RELU)
            between()
            g.gemm_lora_nt(h, W2, down, ids, x, beta=1.0, C=x)
            between()
            if i % 2:
                g.gemm_lora_nt(y, W1, up, ids, h)      # the same buffers with nothing in between
                g.gemm_lora_nt(h, W2, down, ids, y)
                between()
                x.add_(y)
                between()

    layers(torch.cuda.synchronize)
    want = x.clone()
    assert bool(want.isfinite().all())
    for _ in range(5):
        layers(lambda: None)
        assert torch.equal(x, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layers(lambda: None)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layers(lambda: None)
        for _ in range(5):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    g.gemm_f16_nt_check(device=DEV)


def test_no_factors_no_adapters_and_empty():
    X, lora, ids, gen = draw(6, 64, 128, 8, 3, torch.float16, 5)
    one = g.Lora(lora.A, lora.B)
    ref, err = delta64(X, one, ids)
    check(g.gemm_lora_delta(X, one, ids), ref, 1.01 * UNIT[torch.float16] * ref.abs() + err + FLOOR)
    W, C = (torch.randn(s, generator=gen, device=DEV).half() for s in ((64, 128), (6, 64)))
    empty = g.Lora(lora.A[:0], lora.B[:0])
    D, P = torch.empty(6, 64, dtype=torch.float16, device=DEV), torch.empty(6, 64, dtype=torch.float16, device=DEV)
    g.gemm_lora_nt(X, W, empty, ids, D, beta=0.3, C=C)
    g.gemm_nt_ex(X, W, P, beta=0.3, C=C)
    assert torch.equal(D, P)
    assert not bool(g.gemm_lora_delta(X, empty, ids).any())
    assert torch.equal(g.gemm_lora_delta(X, empty, ids, beta=1.0, C=C), C)
    assert g.gemm_lora_delta(X[:0], lora, ids[:0]).shape == (0, 64)
    k0 = g.Lora(lora.A[:, :, :0].contiguous(), lora.B)
    assert torch.equal(g.gemm_lora_delta(X[:, :0].contiguous(), k0, ids, beta=2.0, C=C), C * 2)
    g.gemm_lora_nt(X[:, :0].contiguous(), W[:, :0].contiguous(), k0, ids, D, beta=2.0, C=C)
    assert torch.equal(D, C * 2)


def test_nothing_is_written_beyond_the_rows():
    M, N = 5, 40
    X, lora, ids, _ = draw(M, N, 128, 8, 3, torch.bfloat16, 6)
    wide = torch.full((M + 4, N), 3.0, dtype=torch.bfloat16, device=DEV)
    g.gemm_lora_delta(X, lora, ids, wide[:M])
    assert bool((wide[M:] == 3.0).all()) and bool((wide[:M] != 3.0).any())


def test_streams_and_captured_calls():
    """Two streams at one time, and replays with other ids and activations."""
    N, K = 520, 1024
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i, s in enumerate(streams):
        X, lora, ids, gen = draw(70 + 200 * i, N, K, 16, 5, torch.bfloat16, i)
        W = (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).bfloat16()
        D = torch.empty(len(X), N, dtype=torch.bfloat16, device=DEV)
        g.gemm_lora_nt(X, W, lora, ids, D, stream=s)
        work.append((X, W, lora, ids, D, gen))
    torch.cuda.synchronize()
    want = [w[4].clone() for w in work]
    for _ in range(20):
        for (X, W, lora, ids, D, _), s in zip(work, streams):
            g.gemm_lora_nt(X, W, lora, ids, D, stream=s)
    torch.cuda.synchronize()
    for w, ref in zip(work, want):
        assert torch.equal(w[4], ref)
    X, W, lora, ids, D, gen = work[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        g.gemm_lora_nt(X, W, lora, ids, D)
    for _ in range(3):
        X.copy_(torch.randn(X.shape, generator=gen, device=DEV))
        ids.copy_(torch.randint(-1, 5, ids.shape, generator=gen, device=DEV))
        graph.replay()
    torch.cuda.synchronize()
    E = torch.empty_like(D)
    g.gemm_lora_nt(X, W, lora, ids, E)
    assert torch.equal(D, E)
    g.gemm_f16_nt_check(device=DEV)


def test_refusals():
    X, lora, ids, _ = draw(4, 64, 128, 8, 3, torch.float16, 1)
    W, D = torch.zeros(64, 128, dtype=torch.float16, device=DEV), torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    A, B, f = lora.A, lora.B, lora.factors
    for error, change in [
            (TypeError, dict(X=X.float())), (ValueError, dict(X=X[:, :64])), (TypeError, dict(lora=(A, B))),
            (ValueError, dict(lora=g.Lora(A[:2], B, f))), (ValueError, dict(lora=g.Lora(A, B[:, :, :4].contiguous(), f))),
            (TypeError, dict(lora=g.Lora(A.bfloat16(), B, f))), (TypeError, dict(lora=g.Lora(A, B, f.double()))),
            (ValueError, dict(lora=g.Lora(A, B, f[:2]))), (TypeError, dict(ids=ids.long())), (ValueError, dict(ids=ids[:3])),
            (ValueError, dict(ids=ids.cpu())), (ValueError, dict(W=W[:32])), (TypeError, dict(D=D.bfloat16())),
            (ValueError, dict(D=D[:2])), (g.GemmError, dict(beta=1.0)),
            (g.GemmError, dict(lora=g.Lora(A[:, :4].contiguous(), B[:, :, :4].contiguous(), f)))]:
        args = dict(X=X, W=W, lora=lora, ids=ids, D=D) | change
        with pytest.raises(error):
            g.gemm_lora_nt(**args)
        if "W" in change:
            continue
        args.pop("W")
        args["U"] = args.pop("D")
        with pytest.raises(error):
            g.gemm_lora_delta(**args)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,four", [(8, True), (13, True), (40, True), (64, True), (300, True), (24, False), (64, False), (130, False), (600, False)])
def test_rows_without_an_adapter(M, four, dtype):
    """The plain product's bits with beta 1, or 0 without a bias; with a bias and beta 0 up to one more rounding in fp32."""
    N, K = 1032, 1024
    X, lora, ids, gen = draw(M, N, K, 16, 6, dtype, M)
    W = random_w4(torch.Generator().manual_seed(M), (), N, K, 64, True, dtype, DEV) if four else \
        (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).to(dtype)
    product = g.gemm_w4_nt if four else g.gemm_nt_ex
    C, bias = (torch.randn(s, generator=gen, device=DEV).to(dtype) for s in ((M, N), (N,)))
    sn = torch.rand(N, generator=gen, device=DEV) + 0.5
    ids[1::3] = -1
    none = ids < 0
    D, P = (torch.empty(M, N, dtype=dtype, device=DEV) for _ in range(2))
    for args in (dict(), dict(alpha=0.6, scale_n=sn), dict(alpha=0.6, activation=g.Activation.RELU),
                 dict(alpha=0.6, scale_n=sn, beta=1.0, C=C, bias=bias, activation=g.Activation.RELU)):
        g.gemm_lora_nt(X, W, lora, ids, D, **args)
        product(X, W, P, **args)
        assert torch.equal(D[none], P[none])
    args = dict(alpha=0.6, scale_n=sn, bias=bias)
    g.gemm_lora_nt(X, W, lora, ids, D, **args)
    product(X, W, P, **args)
    d, p = D[none].double(), P[none].double()
    # two fp32 sums that differ in the rounding of one product and of the whole, each then rounded to the type
    x = (p - bias.double()).abs()
    assert bool(((d - p).abs() <= 2.02 * UNIT[dtype] * p.abs() + 2.0 ** -22 * (x + bias.double().abs()) + 2 * FLOOR).all())


def test_adapters_that_nobody_uses():
    """A stack with more adapters may share K out in another way: sums change by their roundings and no more."""
    X, lora, ids, _ = draw(64, 1032, 4096, 64, 4, torch.bfloat16, 22)
    more = g.Lora(torch.cat([lora.A] * 20), torch.cat([lora.B] * 20), torch.cat([lora.factors] * 20))
    ref, err = delta64(X, lora, ids)
    for l in (lora, more):
        check(g.gemm_lora_delta(X, l, ids), ref, 1.01 * UNIT[torch.bfloat16] * ref.abs() + err + FLOOR)


# by the rule that shares rows out, on 152 SMs: clusters of 3, 1, 3, 3, 1 and 1 CTAs for up to 256 rows; with units
# of 32 rows clusters of 1, 3, 8, 6, 3, 1 and 4, of 64 rows of 3, of 128 rows of 6
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,R,count", [(200, 1032, 1032, 8, 105), (256, 264, 1032, 8, 900), (180, 520, 1032, 24, 105), (40, 1032, 520, 40, 200),
                                           (150, 520, 1032, 40, 200), (150, 520, 264, 256, 200),
                                           (300, 520, 1032, 16, 500), (257, 1032, 520, 40, 44), (300, 1032, 1032, 256, 3),
                                           (700, 520, 2056, 136, 1), (260, 264, 520, 200, 44), (500, 520, 264, 256, 300),
                                           (1000, 1032, 520, 144, 5), (4096, 264, 520, 8, 64), (2000, 264, 520, 64, 8)])
def test_ways_to_share_the_rows(M, N, K, R, count, dtype):
    for runs in (False, True):
        X, lora, ids, gen = draw(M, N, K, R, count, dtype, M + N + R, runs)
        C = torch.randn(M, N, generator=gen, device=DEV).to(dtype)
        ref, err = delta64(X, lora, ids, 0.3, C)
        U = g.gemm_lora_delta(X, lora, ids, beta=0.3, C=C)
        check(U, ref, 1.01 * UNIT[dtype] * ref.abs() + err + FLOOR)
        assert torch.equal(g.gemm_lora_delta(X, lora, ids, beta=0.3, C=C), U)
    g.gemm_f16_nt_check(device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,R", [(9, 16), (40, 16), (40, 64), (200, 32), (300, 16), (300, 136)])
def test_not_a_number_reaches_its_row(M, R, dtype):
    """A NaN in a row whose adapter is in use makes that row NaN, whatever the other rows of the adapter hold."""
    X, lora, ids, _ = draw(M, 264, 512, R, 4, dtype, 21, none=0.0)
    want = g.gemm_lora_delta(X, lora, ids)
    rows = [3, M - 2]
    X[rows[0], 0] = X[rows[1], 511] = float("nan")
    got = g.gemm_lora_delta(X, lora, ids)
    assert bool(got[rows].isnan().all())
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert torch.equal(got[keep], want[keep])
