"""The stream-K small-M kernel's workspace (needs a GB300): a workspace that a larger
problem outgrows stays whole for whatever still uses it."""
import threading

import pytest

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

STREAMK = g.Variant.SKINNY_STREAMK
# workspaces from small to large
SHAPES = [(16, 1024, 1024), (16, 4096, 2048), (32, 8192, 1024), (64, 8192, 2048), (64, 16384, 1024)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


def _operands(M, N, K, seed):
    """Whole numbers: every order of summation gives the same exact result."""
    gen = torch.Generator().manual_seed(seed)
    A, B = (torch.randint(-1, 2, (n, K), generator=gen).half().cuda() for n in (M, N))
    return A, B, (A.float() @ B.float().t()).half()


def test_a_captured_call_outlives_a_larger_one():
    torch.backends.cuda.matmul.allow_tf32 = False
    s = torch.cuda.Stream()
    A, B, want = _operands(*SHAPES[0], 1)
    D = torch.empty_like(want)
    torch.cuda.synchronize()
    g.gemm_f16_nt_variant(A, B, D, variant=STREAMK, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.gemm_f16_nt_variant(A, B, D, variant=STREAMK, stream=s)
    for shape in SHAPES[1:]:
        a, b, w = _operands(*shape, 2)
        d = torch.empty_like(w)
        torch.cuda.synchronize()
        g.gemm_f16_nt_variant(a, b, d, variant=STREAMK, stream=s)
        s.synchronize()
        assert torch.equal(d, w)
        D.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        g.gemm_f16_nt_check(stream=s)
        assert torch.equal(D, want)


def test_two_threads_grow_one_workspace():
    torch.backends.cuda.matmul.allow_tf32 = False
    s = torch.cuda.Stream()
    work = [[(*_operands(*shape, 10 * i + n), shape) for n, shape in enumerate(SHAPES)] for i in range(2)]
    outs = [[torch.empty_like(w[2]) for w in ws] for ws in work]
    torch.cuda.synchronize()
    gate = threading.Barrier(2)
    errors = []

    def run(i):
        try:
            for (a, b, _, _), d in zip(work[i], outs[i]):
                gate.wait(60)
                for _ in range(5):
                    g.gemm_f16_nt_variant(a, b, d, variant=STREAMK, stream=s)
        except BaseException as e:   # noqa: B902  (reported by the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    g.gemm_f16_nt_check(stream=s)
    for ws, ds in zip(work, outs):
        for (_, _, want, shape), d in zip(ws, ds):
            assert torch.equal(d, want), shape


PER_THREAD = 2   # the handle cudaStreamPerThread


def test_the_per_thread_stream_has_a_workspace_in_every_thread():
    torch.backends.cuda.matmul.allow_tf32 = False
    shapes = [(16, 8192, 4096), (64, 8192, 4096), (33, 4096, 8192)]   # long enough to run side by side
    work = [_operands(*shape, i) for i, shape in enumerate(shapes)]
    outs = [[torch.empty_like(w[2]) for _ in range(40)] for w in work]
    torch.cuda.synchronize()
    gate = threading.Barrier(len(work))
    errors = []

    def run(i):
        try:
            gate.wait(60)
            for d in outs[i]:
                g.gemm_f16_nt_variant(work[i][0], work[i][1], d, variant=STREAMK, stream=PER_THREAD)
        except BaseException as e:   # noqa: B902  (reported by the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    torch.cuda.synchronize()
    g.gemm_f16_nt_check(device=work[0][0].device)
    for w, ds, shape in zip(work, outs, shapes):
        assert all(torch.equal(d, w[2]) for d in ds), shape
