"""The C entry points of the norm, the row-scaled product and the adapters on the
host (no GPU): what they refuse before any device call."""
import ctypes

import pytest

import dense_fp16_gemm_f16_gb300 as g
from dense_fp16_gemm_f16_gb300 import build as gbuild
from dense_fp16_gemm_f16_gb300.llm import LoraStack, NormOut, Weights

P = 0x7F0000000000          # 16-byte aligned addresses that are never dereferenced here
GAP = 1 << 36
A, B, C, D, E, F, G = (P + i * GAP for i in range(7))
S = g.Status
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return g.load()


def test_norm_refusals(lib):
    def call(dtype=1, X=A, r=B, w=C, eps=1e-6, T=4, H=64, Y=D, Y8=E, scales=F, total=G, kind=2, scale=0.0, out=True):
        o = ctypes.byref(NormOut(Y, Y8, scales, total, kind, scale)) if out else None
        return lib.gemm_rmsnorm(dtype, X, r, w, eps, T, H, o, None)
    for bad in (dict(dtype=2), dict(dtype=-1), dict(T=-1), dict(H=-8), dict(T=2 ** 31), dict(H=2 ** 31), dict(out=False),
                dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(Y=None, Y8=None, scales=None), dict(kind=0), dict(kind=4),
                dict(scales=None), dict(scale=0.5), dict(scales=None, scale=-0.5), dict(scales=None, scale=NAN),
                dict(scales=None, scale=INF), dict(Y8=None), dict(Y8=None, scales=None, scale=1.0), dict(X=0),
                dict(Y=A + 64), dict(total=B + 64), dict(Y=C), dict(Y8=A), dict(Y8=B + 256), dict(scales=A), dict(scales=C),
                dict(total=D), dict(total=D + 128), dict(Y8=D), dict(scales=E + 16), dict(scales=G), dict(Y=A, total=A)):
        assert call(**bad) == S.ERR_INVALID_VALUE, bad
    for bad in (dict(H=60), dict(X=A + 8), dict(r=B + 2), dict(w=C + 8), dict(Y=D + 8), dict(Y8=E + 8), dict(scales=F + 2),
                dict(total=G + 2)):
        assert call(**bad) == S.ERR_MISALIGNED, bad
    for nothing in (dict(T=0), dict(H=0), dict(T=0, Y=None)):
        assert call(**(dict(X=0, r=0, w=0) | nothing)) == S.OK


def test_scaled_product_refusals(lib):
    def call(dtype=2, a=A, sm=B, b=C, d=D, M=4, N=64, K=64, epi=None):
        return lib.gemm_nt_scaled(dtype, a, sm, b, d, M, N, K, epi, None)
    for bad in (dict(dtype=0), dict(dtype=1), dict(dtype=4), dict(sm=0), dict(sm=D), dict(sm=D + 16), dict(M=-1), dict(a=0),
                dict(b=0), dict(d=0), dict(d=A), dict(M=2 ** 31)):
        assert call(**bad) == S.ERR_INVALID_VALUE, bad
    for bad in (dict(sm=B + 2), dict(K=72), dict(N=12), dict(a=A + 8)):
        assert call(**bad) == S.ERR_MISALIGNED, bad
    epi = g.Epilogue(1.0, 1.0, None, None, 0, 0, None)
    assert call(epi=ctypes.byref(epi)) == S.ERR_INVALID_VALUE   # beta without C
    assert call(M=0, a=0, d=0, sm=0) == S.OK
    assert call(N=0, b=0, d=0, sm=0) == S.OK


def _lora(a=B, b=C, f=D, count=4, R=16):
    return ctypes.byref(LoraStack(a, b, f, count, R))


def test_adapter_refusals(lib):
    def delta(dtype=0, X=A, l=None, ids=E, beta=0.0, c=None, U=F, M=4, N=64, K=64):
        return lib.gemm_lora_delta(dtype, X, l or _lora(), ids, beta, c, U, M, N, K, None)

    def nt(dtype=0, X=A, l=None, ids=E, U=F, M=4, N=64, K=64, w=None, epi=None):
        return lib.gemm_lora_nt(dtype, X, w or ctypes.byref(Weights(G, None, None, 0, 0)), l or _lora(), ids, U, M, N, K, epi, None)

    assert lib.gemm_lora_delta(0, A, None, E, 0.0, None, F, 4, 64, 64, None) == S.ERR_INVALID_VALUE
    assert lib.gemm_lora_nt(0, A, None, _lora(), E, F, 4, 64, 64, None, None) == S.ERR_INVALID_VALUE
    for f in (delta, nt):
        for bad in (dict(dtype=2), dict(M=-1), dict(N=-8), dict(K=-8), dict(M=2 ** 31), dict(X=0), dict(U=0), dict(ids=0),
                    dict(l=_lora(a=0)), dict(l=_lora(b=0)), dict(l=_lora(count=-1)), dict(l=_lora(R=0)), dict(l=_lora(R=264)),
                    dict(U=A), dict(U=B + 64), dict(U=C), dict(U=D), dict(U=E),
                    dict(l=_lora(count=2 ** 31 - 1, R=256), K=2 ** 30, N=8)):
            assert f(**bad) == S.ERR_INVALID_VALUE, bad
        for bad in (dict(K=60), dict(N=12), dict(l=_lora(R=12)), dict(X=A + 8), dict(U=F + 8), dict(ids=E + 2),
                    dict(l=_lora(a=B + 8)), dict(l=_lora(b=C + 2)), dict(l=_lora(f=D + 2))):
            assert f(**bad) == S.ERR_MISALIGNED, bad
        assert f(M=0, X=0, U=0, ids=0) == S.OK
        assert f(N=0, U=0) == S.OK
    assert delta(beta=1.0) == S.ERR_INVALID_VALUE            # beta without C
    assert delta(beta=1.0, c=F + 64) == S.ERR_INVALID_VALUE  # partly over U
    assert nt(U=G) == S.ERR_INVALID_VALUE
    assert nt(w=ctypes.byref(Weights(G, D, None, 48, 0))) == S.ERR_INVALID_VALUE
    epi = g.Epilogue(1.0, 1.0, None, None, 0, 0, None)
    assert nt(epi=ctypes.byref(epi)) == S.ERR_INVALID_VALUE
