"""The mixture-of-experts products at the ends of their ranges, on a GB300 against
the 64-bit form: experts whose matrices are too large to be read twice from L2 (the
kernels then take all of an expert's tokens at once), the most choices and experts,
rows too long for their columns to stay in shared memory."""
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


def _run(X, E, k, W13, W2, gen):
    T = X.shape[0]
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32).cuda()
    weights = torch.rand((T, k), generator=gen).cuda()
    Y = torch.full_like(X, float("nan"))
    g.gemm_moe_ffn(X, ids, weights, W13, W2, Y)
    g.gemm_f16_nt_check(device=X.device)
    lc.check(Y, *lc.ffn64(X, ids, weights, W13, W2), f"{T} tokens")


def test_experts_of_16_bits():
    H, I, E = 4096, 3208, 2
    gen = torch.Generator().manual_seed(1)
    W13 = (torch.randn((E, 2 * I, H), generator=gen) / H ** 0.5).bfloat16().cuda()
    W2 = (torch.randn((E, H, I), generator=gen) / I ** 0.5).bfloat16().cuda()
    for T in (3, 12, 30, 64):
        for k in (1, 2):
            _run(torch.randn((T, H), generator=gen).bfloat16().cuda(), E, k, W13, W2, gen)


def test_experts_of_4_bits():
    H, I, E = 8192, 6400, 1
    gen = torch.Generator().manual_seed(2)
    W13 = lc.random_w4(gen, (E,), 2 * I, H, 64, True, torch.float16)
    W2 = lc.random_w4(gen, (E,), H, I, 128, False, torch.float16)
    for T in (2, 6, 17, 40, 64):
        _run(torch.randn((T, H), generator=gen).half().cuda(), E, 1, W13, W2, gen)


# kinds: 0 = 16-bit, a group = 4-bit symmetric, minus a group = 4-bit with zero points
@pytest.mark.parametrize("kind", [0, -32, 128])
@pytest.mark.parametrize("T,H,I,E,k", [(64, 256, 128, 1024, 16), (64, 384, 256, 64, 16), (64, 256, 384, 16, 16), (64, 16384, 128, 4, 2),
                                       (10, 128, 16384, 3, 2), (64, 128, 128, 1024, 1)])
def test_ends_of_the_ranges(T, H, I, E, k, kind):
    gen = torch.Generator().manual_seed(T + H + I + E + k)

    def one(rows, K):
        if kind == 0:
            return (torch.randn((E, rows, K), generator=gen) / K ** 0.5).bfloat16().cuda()
        return lc.random_w4(gen, (E,), rows, K, abs(kind), kind < 0, torch.bfloat16)
    W13, W2 = one(2 * I, H), one(H, I)
    _run(torch.randn((T, H), generator=gen).bfloat16().cuda(), E, k, W13, W2, gen)
