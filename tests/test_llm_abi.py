"""The C entry points of the 4-bit-weight and mixture-of-experts operators on
the host (no GPU): what they refuse before any device call."""
import ctypes

import pytest

import dense_fp16_gemm_f16_gb300 as g
from dense_fp16_gemm_f16_gb300 import build as gbuild
from dense_fp16_gemm_f16_gb300.llm import Weights

P = 0x7F0000000000          # 16-byte aligned addresses that are never dereferenced here
GAP = 1 << 36
A, B, C, D, E, F = (P + i * GAP for i in range(6))
S = g.Status


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return g.load()


def _w4(data=B, scales=C, zeros=None, group=32):
    return ctypes.byref(Weights(data, scales, zeros, group, 0))


def test_quantize_refusals(lib):
    def call(dtype=0, W=A, batch=1, N=64, K=64, group=32, codes=B, scales=C, zeros=D):
        return lib.gemm_w4_quantize(dtype, W, batch, N, K, group, codes, scales, zeros, None)
    for bad in (dict(dtype=2), dict(dtype=-1), dict(N=-8), dict(K=-32), dict(batch=-1), dict(group=16), dict(group=0),
                dict(batch=2 ** 31), dict(batch=2 ** 20, N=2 ** 20), dict(W=0), dict(codes=0), dict(scales=0),
                dict(codes=A), dict(scales=A + 64), dict(zeros=C), dict(scales=B + 16)):
        assert call(**bad) == S.ERR_INVALID_VALUE, bad
    for bad in (dict(K=48), dict(N=12), dict(W=A + 8), dict(codes=B + 4), dict(scales=C + 2), dict(zeros=D + 8)):
        assert call(**bad) == S.ERR_MISALIGNED, bad
    for nothing in (dict(batch=0), dict(N=0), dict(K=0)):
        assert call(W=0, codes=0, scales=0, zeros=0, **nothing) == S.OK


def test_dequantize_refusals(lib):
    def call(w=None, dtype=0, batch=1, N=64, K=64, W=A):
        return lib.gemm_w4_dequantize(dtype, w or _w4(), batch, N, K, W, None)
    assert lib.gemm_w4_dequantize(0, None, 1, 64, 64, A, None) == S.ERR_INVALID_VALUE
    assert call(_w4(scales=None)) == S.ERR_INVALID_VALUE
    assert call(_w4(group=48)) == S.ERR_INVALID_VALUE
    assert call(W=0) == S.ERR_INVALID_VALUE
    assert call(W=B) == S.ERR_INVALID_VALUE
    assert call(N=4) == S.ERR_MISALIGNED
    assert call(W=A + 2) == S.ERR_MISALIGNED
    assert call(batch=0, W=0) == S.OK


def test_product_refusals(lib):
    def call(w=None, dtype=1, M=4, N=64, K=64, a=A, d=D, epi=None):
        return lib.gemm_w4_nt(dtype, a, w or _w4(), d, M, N, K, epi, None)
    assert call(dtype=2) == S.ERR_INVALID_VALUE
    assert call(M=-1) == S.ERR_INVALID_VALUE
    assert call(M=2 ** 31) == S.ERR_INVALID_VALUE
    assert call(a=0) == S.ERR_INVALID_VALUE
    assert call(d=0) == S.ERR_INVALID_VALUE
    assert call(d=A) == S.ERR_INVALID_VALUE
    assert call(d=C) == S.ERR_INVALID_VALUE            # over the scales
    assert call(_w4(zeros=D + 64)) == S.ERR_INVALID_VALUE
    assert call(_w4(scales=None, group=0)) == S.ERR_INVALID_VALUE
    assert call(K=80) == S.ERR_MISALIGNED
    assert call(N=20) == S.ERR_MISALIGNED
    assert call(a=A + 8) == S.ERR_MISALIGNED
    epi = g.Epilogue(1.0, 1.0, None, None, 0, 0, None)
    assert call(epi=ctypes.byref(epi)) == S.ERR_INVALID_VALUE   # beta without C
    epi = g.Epilogue(1.0, 0.0, None, E + 2, 0, 0, None)
    assert call(epi=ctypes.byref(epi)) == S.ERR_MISALIGNED
    assert call(M=0, a=0, d=0) == S.OK
    assert call(N=0, a=0, d=0) == S.OK


def test_route_refusals(lib):
    def call(dtype=0, X=A, Wr=B, bias=None, T=4, H=64, E=8, k=2, scoring=0, ids=C, w=D):
        return lib.gemm_moe_route(dtype, X, Wr, bias, T, H, E, k, scoring, 1, ids, w, None)
    for bad in (dict(dtype=3), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=32, k=17),
                dict(scoring=2), dict(X=0), dict(Wr=0), dict(ids=0), dict(w=0), dict(ids=A), dict(w=B), dict(w=C),
                dict(bias=D)):
        assert call(**bad) == S.ERR_INVALID_VALUE, bad
    for bad in (dict(H=60), dict(X=A + 8), dict(Wr=B + 2), dict(ids=C + 4), dict(bias=F + 4)):
        assert call(**bad) == S.ERR_MISALIGNED, bad
    assert call(T=0, X=0, Wr=0, ids=0, w=0) == S.OK


def test_ffn_and_layer_refusals(lib):
    w16 = lambda p: ctypes.byref(Weights(p, None, None, 0, 0))   # noqa: E731

    def call(dtype=0, X=A, ids=B, w=C, w13=None, w2=None, Y=F, T=4, H=64, I=32, E_=8, k=2):
        return lib.gemm_moe_ffn(dtype, X, ids, w, w13 or w16(D), w2 or w16(E), Y, T, H, I, E_, k, None)

    def layer(X=A, Wr=B, w13=None, w2=None, Y=F, T=4, H=64, I=32, E_=8, k=2, scoring=0):
        return lib.gemm_moe_layer(0, X, Wr, None, w13 or w16(D), w2 or w16(E), Y, T, H, I, E_, k, scoring, 1, None)

    for f in (call, layer):
        for bad in (dict(T=-1), dict(T=65), dict(I=0), dict(H=0), dict(E_=0), dict(k=0), dict(k=17), dict(X=0), dict(Y=0),
                    dict(Y=A), dict(Y=D + 64), dict(Y=E), dict(w13=w16(0)),
                    dict(w13=ctypes.byref(Weights(D, None, C, 0, 0))), dict(w2=ctypes.byref(Weights(D, None, None, 32, 0))),
                    dict(w2=ctypes.byref(Weights(D, C, None, 33, 0)))):
            assert f(**bad) == S.ERR_INVALID_VALUE, bad
        for bad in (dict(H=60), dict(I=20), dict(X=A + 8), dict(Y=F + 2), dict(w13=w16(D + 8)),
                    dict(I=40, w2=ctypes.byref(Weights(D, C, None, 32, 0)))):
            assert f(**bad) == S.ERR_MISALIGNED, bad
        assert f(T=0, X=0, Y=0) == S.OK
    assert call(dtype=2) == S.ERR_INVALID_VALUE
    assert call(ids=0) == S.ERR_INVALID_VALUE
    assert call(w=0) == S.ERR_INVALID_VALUE
    assert call(ids=F) == S.ERR_INVALID_VALUE
    assert call(w=C + 4) == S.ERR_MISALIGNED
    assert layer(scoring=5) == S.ERR_INVALID_VALUE
    assert layer(Wr=F) == S.ERR_INVALID_VALUE
