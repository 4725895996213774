"""Outputs that a call allocates itself, on a stream that is not the current one (needs a GB300)."""
import pytest

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PAUSE = 40_000_000   # clocks: about 20 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


def _calls():
    """name -> call(stream) that returns its outputs as a list."""
    gen = torch.Generator().manual_seed(1)
    W = torch.randn((1024, 2048), generator=gen).half().cuda()
    X, Wr = torch.randn((64, 512), generator=gen).half().cuda(), torch.randn((32, 512), generator=gen).div_(16).half().cuda()
    packed = g.gemm_w4_quantize(W, 64, symmetric=False)

    def pack(s):
        out = g.gemm_w4_quantize(W, 64, symmetric=False, stream=s)
        return [out.codes, out.scales, out.zeros]

    return {"pack": pack, "unpack": lambda s: [g.gemm_w4_dequantize(packed, stream=s)],
            "route": lambda s: list(g.gemm_moe_route(X, Wr, k=4, stream=s)), "gemm": lambda s: [g.gemm(X, Wr, stream=s)]}


def _ways(s):
    return {"stream": s, "handle": s.cuda_stream}


@pytest.mark.parametrize("name", ["pack", "unpack", "route", "gemm"])
@pytest.mark.parametrize("way", ["stream", "handle"])
def test_work_queued_on_the_current_stream_does_not_reach_them(name, way):
    call = _calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    for t in want:   # blocks of the same sizes, written late and free by now
        late = [torch.empty_like(t) for _ in range(4)]
        for x in late:
            x.view(torch.uint8).fill_(0xEE)
        del late, x
    got = call(_ways(s)[way])
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["pack", "unpack", "route", "gemm"])
@pytest.mark.parametrize("way", ["stream", "handle"])
def test_dropped_early_they_are_not_given_away(name, way):
    call = _calls()[name]
    shapes = [(t.shape, t.dtype) for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)
    call(_ways(s)[way])   # dropped while its kernel still waits
    mine = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((t == 0).all()) for t in mine)


@pytest.mark.parametrize("name", ["pack", "unpack", "route", "gemm"])
def test_dropped_by_the_current_stream_they_are_not_given_away(name):
    call = _calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(PAUSE)
    kept = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(s):
        over = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and len(over) == 4 * len(want)


def test_default_and_per_thread_streams():
    call = _calls()["route"]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for default in (0, 1):
            got = call(default)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError):
        call(2)
