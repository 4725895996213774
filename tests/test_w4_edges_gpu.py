"""4-bit packing where scales are the smallest numbers of their type, on a GB300."""
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


# largest scales of a group: the last normal numbers, the subnormal ones whose reciprocal
# is still finite, and those whose reciprocal is not (bf16 only), down to zero
SCALES = {"f16": (torch.float16, range(-26, -12)), "bf16": (torch.bfloat16, range(-136, -122))}


@pytest.mark.parametrize("dtype", SCALES)
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group", [32, 128])
def test_quantize_of_the_smallest_scales(dtype, asym, group):
    dtype, exponents = SCALES[dtype]
    gen = torch.Generator().manual_seed(group)
    rows = []
    for e in exponents:
        for kind in range(4):
            w = torch.randint(-7, 8, (group,), generator=gen).double()            # whole steps, with zeros
            if kind == 1:
                w = torch.rand((group,), generator=gen).double() * 15 - 6           # any values
            elif kind == 2:
                w = (w * 2).clamp(-7, 7) / 2 + 0.25                                 # steps and a half, and the like
            elif kind == 3:
                w = w.abs()                                                        # no negative weight
            w[0] = 7.0 if not asym or kind != 1 else 9.0
            rows.append(w * 2.0 ** e)
    W = torch.stack(rows).to(dtype)
    W = torch.cat((W, W.flip(1)), 1).contiguous()                                 # two groups a row
    out = g.gemm_w4_quantize(W.cuda(), group, symmetric=not asym)
    codes, scales, zeros = lc.quantize64(W, group, asym)
    assert torch.equal(out.scales.cpu(), scales.contiguous())
    if asym:
        assert torch.equal(out.zeros.cpu(), zeros.contiguous())
    assert torch.equal(out.codes.cpu(), codes)
    values = g.gemm_w4_dequantize(out).cpu()
    on_host = g.W4(codes, scales.contiguous(), None if zeros is None else zeros.contiguous(), group)
    assert torch.equal(values, lc.w64(on_host)[0].float().to(dtype))
