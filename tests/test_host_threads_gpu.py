"""The entry points from a host thread that has made no CUDA call yet (needs a GB300).

The CUDA runtime makes a device's context current in a thread at the thread's first
call that needs it.  Encoding a tensor map needs a current context but does not bring
one, so the library has to."""
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


def _in_new_thread(call):
    errors = []

    def work():
        try:
            call()
        except BaseException as e:   # noqa: B902  (reported by the test's thread)
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join(60)
    assert not errors, errors
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [8, 512])
def test_dense_products(M):
    gen = torch.Generator().manual_seed(M)
    A, B = (torch.randn((n, 256), generator=gen).half().cuda() for n in (M, 384))
    want, got = (torch.full((M, 384), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    g.gemm_f16_nt(A, B, want)
    torch.cuda.synchronize()
    _in_new_thread(lambda: g.gemm_f16_nt(A, B, got))
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [4, 100])
def test_4_bit_products(M):
    gen = torch.Generator().manual_seed(M)
    A, B = (torch.randn((n, 256), generator=gen).half().cuda() for n in (M, 384))
    W = g.gemm_w4_quantize(B, 32)
    want, got = (torch.full((M, 384), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    g.gemm_w4_nt(A, W, want)
    torch.cuda.synchronize()
    _in_new_thread(lambda: g.gemm_w4_nt(A, W, got))
    assert torch.equal(got, want)


def test_experts():
    gen = torch.Generator().manual_seed(3)
    X = torch.randn((6, 256), generator=gen).half().cuda()
    W13, W2 = (torch.randn(s, generator=gen).div_(16).half().cuda() for s in ((4, 256, 256), (4, 256, 128)))
    ids = torch.randint(0, 4, (6, 2), generator=gen).to(torch.int32).cuda()
    weights = torch.rand((6, 2), generator=gen).cuda()
    want, got = (torch.full_like(X, float("nan")) for _ in range(2))
    g.gemm_moe_ffn(X, ids, weights, W13, W2, want)
    torch.cuda.synchronize()
    _in_new_thread(lambda: g.gemm_moe_ffn(X, ids, weights, W13, W2, got))
    assert torch.equal(got, want)
