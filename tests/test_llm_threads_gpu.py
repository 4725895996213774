"""Mixture-of-experts calls from several host threads on a GB300.

The kernels of one call pass logits, choices and the first product's result to one
another through scratch memory of their stream.  Calls of two threads must never
find each other's values there."""
import os
import subprocess
import sys
import threading

import pytest

import dense_fp16_gemm_f16_gb300 as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    assert torch.cuda.is_available(), "this test needs a CUDA GPU"
    gbuild.build()


class Case:
    """One operator on inputs of its own; call(stream) returns its outputs."""

    def __init__(self, op, T, H, I, E, k, seed):
        gen = torch.Generator().manual_seed(seed)
        self.op, self.k = op, k
        self.X = torch.randn((T, H), generator=gen).half().cuda()
        self.Wr = (torch.randn((E, H), generator=gen) / 16).half().cuda()
        self.W13 = (torch.randn((E, 2 * I, H), generator=gen) / H ** 0.5).half().cuda()
        self.W2 = (torch.randn((E, H, I), generator=gen) / I ** 0.5).half().cuda()
        self.ids = torch.randint(0, E, (T, k), generator=gen).to(torch.int32).cuda()
        self.weights = torch.rand((T, k), generator=gen).cuda()

    def outputs(self):
        if self.op == "route":
            return torch.full_like(self.ids, -7), torch.full_like(self.weights, -7.0)
        return (torch.full_like(self.X, float("nan")),)

    def call(self, out, stream):
        if self.op == "route":
            g.gemm_moe_route(self.X, self.Wr, out[0], out[1], stream=stream)
        elif self.op == "ffn":
            g.gemm_moe_ffn(self.X, self.ids, self.weights, self.W13, self.W2, out[0], stream=stream)
        else:
            g.gemm_moe_layer(self.X, self.Wr, self.W13, self.W2, out[0], self.k, stream=stream)

    def alone(self):
        out = self.outputs()
        self.call(out, None)
        torch.cuda.synchronize()
        return out


def _run_threads(cases, streams, calls):
    """Every case from a thread of its own, `calls` times; all outputs against a call alone."""
    want = [c.alone() for c in cases]
    outs = [[c.outputs() for _ in range(calls)] for c in cases]
    torch.cuda.synchronize()
    gate = threading.Barrier(len(cases))
    errors = []

    def work(i):
        try:
            gate.wait(60)
            for out in outs[i]:
                cases[i].call(out, streams[i])
        except BaseException as e:   # noqa: B902  (reported by the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join(120)
    finally:
        sys.setswitchinterval(before)
    assert not errors, errors
    torch.cuda.synchronize()
    g.gemm_f16_nt_check(device=cases[0].X.device)
    for i, case in enumerate(cases):
        wrong = sum(not all(torch.equal(a, b) for a, b in zip(out, want[i])) for out in outs[i])
        assert wrong == 0, f"{case.op} {i}: {wrong} of {calls} calls differ from a call alone"


@pytest.mark.parametrize("op", ["layer", "ffn", "route"])
def test_two_threads_on_one_stream(op):
    # the same sizes, so that values of the other thread would fit; 16 tokens: choice in a kernel of its own
    cases = [Case(op, 16, 512, 256, 8, 2, seed) for seed in (1, 2)]
    for stream in (None, torch.cuda.Stream()):
        _run_threads(cases, [stream, stream], 200)


def test_threads_with_different_operators_on_one_stream():
    cases = [Case("layer", 4, 256, 128, 8, 2, 3), Case("layer", 64, 512, 384, 16, 4, 4), Case("ffn", 20, 256, 512, 4, 2, 5),
             Case("route", 64, 512, 8, 32, 4, 6)]
    stream = torch.cuda.Stream()
    _run_threads(cases, [stream] * 4, 100)


PER_THREAD = 2   # the handle cudaStreamPerThread


def test_the_per_thread_stream_is_another_stream_in_every_thread():
    # long enough that the threads' kernels run side by side
    cases = [Case("layer", 16, 2048, 1024, 8, 2, seed) for seed in (7, 8, 9)]
    _run_threads(cases, [PER_THREAD] * 3, 60)
    cases = [Case("route", T, 4096, 8, 64, 4, T) for T in (3, 8, 64)]   # up to 8 tokens a counter tells the last CTA
    _run_threads(cases, [PER_THREAD] * 3, 60)


def test_a_destroyed_stream_leaves_its_scratch_to_its_work():
    """A stream that comes after a destroyed one, perhaps with its handle, while the old one's work still waits."""
    a, b = Case("layer", 16, 1024, 512, 8, 2, 11), Case("layer", 16, 1024, 512, 8, 2, 12)
    want = a.alone(), b.alone()
    rt = torch.cuda.cudart()

    def create():
        handle = torch.zeros(1, dtype=torch.int64)
        assert int(rt.cudaStreamCreate(handle.data_ptr())) == 0
        return int(handle)

    for _ in range(4):
        outs = a.outputs(), b.outputs()
        torch.cuda.synchronize()
        first = create()
        with torch.cuda.stream(torch.cuda.ExternalStream(first)):
            torch.cuda._sleep(20_000_000)   # 10 ms: the layer below is still waiting when its stream goes
        a.call(outs[0], first)
        assert int(rt.cudaStreamDestroy(first)) == 0
        second = create()
        b.call(outs[1], second)
        torch.cuda.synchronize()
        assert int(rt.cudaStreamDestroy(second)) == 0
        g.gemm_f16_nt_check(device=a.X.device)
        assert torch.equal(outs[0][0], want[0][0]) and torch.equal(outs[1][0], want[1][0])


# In a process of its own: no stream has had the new one's handle before.
_CAPTURE = """
import torch
import dense_fp16_gemm_f16_gb300 as g
from test_llm_threads_gpu import Case
a = Case("layer", 16, 512, 256, 8, 2, 13)
want = a.alone()[0]
fresh = torch.cuda.Stream()
out = a.outputs()
torch.cuda.synchronize()
refused = False
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=fresh):
        a.call(out, fresh)
except g.GemmError:
    refused = True
assert refused   # no scratch yet; the capture ended well and the stream stays usable
a.call(out, fresh)
torch.cuda.synchronize()
assert torch.equal(out[0], want)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=fresh):
    a.call(out, fresh)
out[0].zero_()
torch.cuda.synchronize()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out[0], want)
print("as expected")
"""


def test_capture_before_and_after_the_first_call_on_a_stream():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    out = subprocess.run([sys.executable, "-c", _CAPTURE], capture_output=True, text=True, timeout=300, env=env)
    assert out.returncode == 0 and "as expected" in out.stdout, out.stdout + out.stderr
