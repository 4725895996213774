"""The norm and the adapters where offsets pass 32 bits, against 64 bits on samples."""
import pytest
import torch

import dense_fp16_gemm_f16_gb300 as g
import test_lora_gpu as lo
import test_norm_gpu as no

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_norm_of_many_rows():
    T, H = 270000, 8192          # 2.2e9 elements
    x = torch.randn(T, H, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(H, device=DEV, dtype=torch.bfloat16)
    total = torch.empty_like(x)
    out = g.gemm_rmsnorm(x, w, x, Y8=g.Dtype.E4M3, total=total)
    at = torch.tensor([0, 1, 131071, 262143, 262144, 262145, T - 2, T - 1], device=DEV)
    no.check(g.Normed(None, out.Y8[at], out.scales[at], None), x[at], x[at], w, 1e-6, H, total[at])


def test_norm_of_a_long_row():
    H = 1 << 27
    x = torch.randn(2, H, device=DEV, dtype=torch.float16)
    out = g.gemm_rmsnorm(x, Y=torch.empty_like(x))
    for t in range(2):
        h = x[t].double()
        y = h / torch.sqrt((h * h).mean() + 1e-6)
        # sums of 2^17 squares in a thread: at most 2^17 roundings of 2^-24, halved by the root
        assert bool(((out.Y[t].double() - y).abs() <= (2.0 ** -8 + 1.01 * 2.0 ** -11) * y.abs() + 2.0 ** -25).all())


def test_adapters_past_32_bits():
    count, R, K, N, M = 700, 64, 49152, 1024, 40      # A: 2.2e9 elements
    gen = torch.Generator(device=DEV).manual_seed(1)
    A = torch.empty(count, R, K, device=DEV, dtype=torch.bfloat16).normal_(generator=gen).mul_(K ** -0.5)
    B = torch.randn(count, N, R, generator=gen, device=DEV, dtype=torch.bfloat16)
    lora = g.Lora(A, B, torch.rand(count, generator=gen, device=DEV))
    for m in (M, 10):
        X = torch.randn(m, K, generator=gen, device=DEV, dtype=torch.bfloat16)
        ids = torch.randint(640, count, (m,), generator=gen, device=DEV, dtype=torch.int32)
        ids[0], ids[1] = count - 1, 0
        ref, err = lo.delta64(X, lora, ids)
        lo.check(g.gemm_lora_delta(X, lora, ids), ref, 1.01 * 2.0 ** -8 * ref.abs() + err + 2.0 ** -25)
        W, D = torch.zeros(N, K, device=DEV, dtype=torch.bfloat16), torch.empty(m, N, device=DEV, dtype=torch.bfloat16)
        g.gemm_lora_nt(X, W, lora, ids, D)
        lo.check(D, ref, 2.02 * 2.0 ** -8 * ref.abs() + 2 * err + 2.0 ** -24)


def test_outputs_past_32_bits():
    M, N, K, R = 300, 8 << 20, 64, 8                  # U: 2.5e9 elements
    X, lora, ids, _ = lo.draw(M, 8, K, R, 2, torch.bfloat16, 2)
    gen = torch.Generator(device=DEV).manual_seed(3)
    B = torch.randn(2, N, R, generator=gen, device=DEV, dtype=torch.bfloat16)
    ids[M - 1], ids[M - 2] = 1, -1
    U = g.gemm_lora_delta(X, g.Lora(lora.A, B, lora.factors), ids)
    cols = torch.tensor([0, 1, 12345, N // 2, N - 1], device=DEV)
    ref, err = lo.delta64(X, g.Lora(lora.A, B[:, cols].contiguous(), lora.factors), ids)
    lo.check(U[:, cols], ref, 1.01 * 2.0 ** -8 * ref.abs() + err + 2.0 ** -25)


def test_more_rows_than_one_list():
    M, N, K, R = 70000, 72, 136, 24
    X, lora, ids, _ = lo.draw(M, N, K, R, 900, torch.float16, 4)
    ref, err = lo.delta64(X, lora, ids)
    lo.check(g.gemm_lora_delta(X, lora, ids), ref, 1.01 * 2.0 ** -11 * ref.abs() + err + 2.0 ** -25)


def test_sum_of_a_long_row_of_one_value():
    """Equal numbers make every rounding of a long sum fall to the same side.  y is 1.  The sum may be off by eight
    roundings of 2^-24 in a piece, two of the pieces' sum and ten between threads, whatever the row's length; the root
    halves that, and the division by H, eps, the root and the product leave four more at most: 14 for y, 15 for the scale."""
    for H in (1 << 24, (1 << 27) + 8):
        for k in (2, 6, 14):
            x = torch.full((2, H), 1.0 + k * 2.0 ** -10, device=DEV, dtype=torch.float16)
            total = torch.empty_like(x)
            out = g.gemm_rmsnorm(x, eps=0.0, Y=torch.empty_like(x), Y8=g.Dtype.E4M3, total=total)
            assert bool(((out.Y.double() - 1.0).abs() <= 1.01 * 2.0 ** -11 + 14 * 2.0 ** -24).all())
            assert bool(((out.scales.double() * 448.0 - 1.0).abs() <= 15 * 2.0 ** -24).all())
            assert torch.equal(total, x) and bool((out.Y8.float() == 448.0).all())
            del out, total


def test_long_rows_of_special_values():
    """A sum of squares beyond fp32's numbers is infinite and its row zero, as in short rows."""
    H = 40000
    x = torch.ones(4, H, device=DEV, dtype=torch.bfloat16)
    x[0] = 2.0 ** 60                    # the sum of one thread's squares is infinite half way
    x[1, 5], x[2, 39999] = float("inf"), float("nan")
    Y = g.gemm_rmsnorm(x).Y
    assert not bool(Y[0].any())
    assert bool(Y[1, 5].isnan()) and int(Y[1].count_nonzero()) == 1
    assert bool(Y[2].isnan().all()) and bool((Y[3] == 1.0).all())
