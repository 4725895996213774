"""4-bit weights and the mixture-of-experts layer: the binding of
``include/gemm_llm.h``.

Tensors are contiguous CUDA tensors on one device; activations, scales, zero
points and outputs are all float16 or all bfloat16.  Calls are asynchronous on
``stream`` (default: the tensors' current stream).  Argument checks happen
here (``TypeError`` / ``ValueError``) and in the library (``GemmError``).

Outputs that are not given are allocated for ``stream``.  A caller that reads them
on another stream waits for ``stream`` first; they may be dropped at any time if
that stream was current at the call, else after ``Tensor.record_stream``.
"""
from __future__ import annotations

import ctypes
import enum

import dense_fp16_gemm_f16_gb300 as _g


class MoeScoring(enum.IntEnum):
    SOFTMAX = 0
    SIGMOID = 1


class Weights(ctypes.Structure):
    """Mirror of gemm_weights_t."""
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class W4:
    """A 4-bit weight matrix [N, K], or a stack of them [E, N, K].

    codes   uint8 [.., N, K/2], the element of even k in the low four bits
    scales  [.., K/group, N] float16 or bfloat16
    zeros   like scales, or None for 8 everywhere
    w[n, k] = scales[k // group, n] * (code[n, k] - zeros[k // group, n])
    """
    __slots__ = ("codes", "scales", "zeros", "group")

    def __init__(self, codes, scales, zeros=None, group: int = 128):
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group

    @property
    def shape(self) -> tuple:
        s = self.codes.shape
        return (*s[:-1], s[-1] * 2)


def declare(lib) -> None:
    p, i64, i32, w = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(Weights)
    for name, args in {
        "gemm_w4_quantize": [i32, p, i64, i64, i64, i32, p, p, p, p],
        "gemm_w4_dequantize": [i32, w, i64, i64, i64, p, p],
        "gemm_w4_nt": [i32, p, w, p, i64, i64, i64, ctypes.POINTER(_g.Epilogue), p],
        "gemm_moe_route": [i32, p, p, p, i64, i64, i64, i32, i32, i32, p, p, p],
        "gemm_moe_ffn": [i32, p, p, p, w, w, p, i64, i64, i64, i64, i32, p],
        "gemm_moe_layer": [i32, p, p, p, w, w, p, i64, i64, i64, i64, i32, i32, i32, p],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_torch = None
_lib = None
_dtypes: dict = {}
_raw_stream = None
_current_device = None


def _setup():
    """torch and the library, once; returns the library."""
    global _torch, _lib, _raw_stream, _current_device
    lib = _g.load()
    import torch
    _dtypes.update({torch.float16: int(_g.Dtype.F16), torch.bfloat16: int(_g.Dtype.BF16)})
    # the current stream's handle without a Stream object around it, which
    # costs 2 us of the 8 that a small call takes
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = torch.cuda.current_device
    _torch, _lib = torch, lib
    return lib


def _type16(t, name: str) -> int:
    try:
        return _dtypes[t.dtype]
    except (KeyError, AttributeError):
        raise TypeError(f"{name} must be a float16 or bfloat16 tensor, got {getattr(t, 'dtype', type(t))}") from None


def _check(t, name: str, dtype, shape, index: int) -> int:
    """The address of a contiguous tensor of this type and shape on CUDA device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not _g._is_tensor(t):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _cuda(t, name: str) -> int:
    """The CUDA device index of a contiguous tensor."""
    if not _g._is_tensor(t):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.get_device()


def _weights(w, name: str, dtype, lead: tuple, N: int, K: int, index: int) -> Weights:
    """A W4 or a 16-bit tensor [*lead, N, K] as the library takes it."""
    if type(w) is not W4:
        return Weights(_check(w, name, dtype, (*lead, N, K), index), None, None, 0, 0)
    group = w.group
    if group not in (32, 64, 128):
        raise ValueError(f"{name}: group must be 32, 64 or 128, got {group}")
    if K % group:
        raise ValueError(f"{name}: K = {K} is not a multiple of the group ({group})")
    side = (*lead, K // group, N)
    return Weights(_check(w.codes, name + ".codes", _torch.uint8, (*lead, N, K // 2), index),
                   _check(w.scales, name + ".scales", dtype, side, index),
                   None if w.zeros is None else _check(w.zeros, name + ".zeros", dtype, side, index), group, 0)


def _run(fn, index: int, stream, args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    if stream is None:
        handle = _raw_stream(index) or None
    else:
        handle = stream.cuda_stream or None if hasattr(stream, "cuda_stream") else int(stream) or None
    if index == _current_device():
        st = fn(*args, handle)
    else:
        with _torch.cuda.device(index):
            st = fn(*args, handle)
    if st:
        raise _g.GemmError(st, fn.__name__)


def gemm_w4_quantize(W, group: int = 128, codes=None, scales=None, zeros=None, symmetric: bool | None = None,
                     stream=None) -> W4:
    """W [N, K] or [E, N, K] in 4 bits with a scale for each `group` of consecutive k.

    ``symmetric`` (default: True unless ``zeros`` is given) uses the fixed zero
    point 8; otherwise every group gets its own.  Outputs are allocated unless given."""
    lib = _lib or _setup()
    index = _cuda(W, "W")
    dt = _type16(W, "W")
    if W.dim() not in (2, 3):
        raise ValueError(f"W must be [N, K] or [E, N, K], got {tuple(W.shape)}")
    *lead, N, K = W.shape
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if K % group:
        raise ValueError(f"K = {K} is not a multiple of the group ({group})")
    if symmetric is None:
        symmetric = zeros is None
    if symmetric and zeros is not None:
        raise ValueError("symmetric weights have no zero points")
    side = (*lead, K // group, N)
    if codes is None:
        codes = _g._empty((*lead, N, K // 2), _torch.uint8, W.device, stream)
    if scales is None:
        scales = _g._empty(side, W.dtype, W.device, stream)
    if zeros is None and not symmetric:
        zeros = _g._empty(side, W.dtype, W.device, stream)
    out = W4(codes, scales, zeros, group)
    w = _weights(out, "output", W.dtype, tuple(lead), N, K, index)
    _run(lib.gemm_w4_quantize, index, stream,
         (dt, W.data_ptr(), lead[0] if lead else 1, N, K, group, w.data, w.scales, w.zeros))
    return out


def gemm_w4_dequantize(W: W4, out=None, stream=None):
    """The float16 / bfloat16 matrices that `W` stands for, in ``out`` (allocated unless given)."""
    lib = _lib or _setup()
    if not isinstance(W, W4):
        raise TypeError("W must be a W4")
    index = _cuda(W.codes, "W.codes")
    dt = _type16(W.scales, "W.scales")
    if W.codes.dim() not in (2, 3):
        raise ValueError(f"W.codes must be [N, K/2] or [E, N, K/2], got {tuple(W.codes.shape)}")
    *lead, N, K = W.shape
    w = _weights(W, "W", W.scales.dtype, tuple(lead), N, K, index)
    if out is None:
        out = _g._empty(W.shape, W.scales.dtype, W.codes.device, stream)
    ptr = _check(out, "out", W.scales.dtype, W.shape, index)
    _run(lib.gemm_w4_dequantize, index, stream,
         (dt, ctypes.byref(w), lead[0] if lead else 1, N, K, ptr))
    return out


def gemm_w4_nt(A, B: W4, D, alpha=1.0, beta=0.0, C=None, bias=None, activation=_g.Activation.NONE, stream=None,
               scale_n=None) -> None:
    """D = act(alpha·scale_n[n]·A·Bᵀ + beta·C + bias[n]) with the weights B [N, K] in 4 bits."""
    lib = _lib or _setup()
    index = _cuda(A, "A")
    dt = _type16(A, "A")
    if not isinstance(B, W4):
        raise TypeError("B must be a W4")
    if A.dim() != 2 or B.codes.dim() != 2:
        raise ValueError("A and B must be matrices")
    M, K = A.shape
    N = B.codes.shape[0]
    dtype = A.dtype
    w = _weights(B, "B", dtype, (), N, K, index)
    d = _check(D, "D", dtype, (M, N), index)
    epi = None
    if alpha != 1.0 or beta != 0.0 or bias is not None or scale_n is not None or activation:
        epi = ctypes.byref(_g.Epilogue(
            float(alpha), float(beta), None if C is None else _check(C, "C", dtype, (M, N), index),
            None if bias is None else _check(bias, "bias", dtype, (N,), index), int(activation), 0,
            None if scale_n is None else _check(scale_n, "scale_n", _torch.float32, (N,), index)))
    _run(lib.gemm_w4_nt, index, stream, (dt, A.data_ptr(), ctypes.byref(w), d, M, N, K, epi))


def _tokens(X, Wr, bias):
    index = _cuda(X, "X")
    dt = _type16(X, "X")
    if X.dim() != 2 or not _g._is_tensor(Wr) or Wr.dim() != 2:
        raise ValueError("X must be [T, H] and Wr [E, H]")
    T, H = X.shape
    E = Wr.shape[0]
    wr = _check(Wr, "Wr", X.dtype, (E, H), index)
    b = None if bias is None else _check(bias, "bias", _torch.float32, (E,), index)
    return index, dt, T, H, E, wr, b


def gemm_moe_route(X, Wr, ids=None, weights=None, k: int | None = None, bias=None, scoring=MoeScoring.SOFTMAX,
                   renormalize: bool = True, stream=None):
    """The k experts of each token and their weights: (ids int32 [T, k], weights float32 [T, k]).

    Scores are softmax or sigmoid of X·Wrᵀ; the k largest logits (with ``bias``
    float32 [E]: the k largest scores + bias) are chosen, largest first, the
    lower expert first where equal.  An id of -1 beside a weight of 0 means that
    no further expert is allowed (bias of minus infinity).  ``k`` is taken from
    ``ids`` where that is given."""
    lib = _lib or _setup()
    index, dt, T, H, E, wr, b = _tokens(X, Wr, bias)
    if k is None:
        if ids is None:
            raise ValueError("give k or ids")
        k = ids.shape[-1]
    if ids is None:
        ids = _g._empty((T, k), _torch.int32, X.device, stream)
    if weights is None:
        weights = _g._empty((T, k), _torch.float32, X.device, stream)
    _run(lib.gemm_moe_route, index, stream,
         (dt, X.data_ptr(), wr, b, T, H, E, k, int(scoring), 1 if renormalize else 0,
          _check(ids, "ids", _torch.int32, (T, k), index),
          _check(weights, "weights", _torch.float32, (T, k), index)))
    return ids, weights


def _experts(W13, W2, dtype, H, E, index):
    """(w13, w2, I) of E experts as the library takes them."""
    rows = W13.codes if isinstance(W13, W4) else W13
    if not _g._is_tensor(rows) or rows.dim() != 3 or rows.shape[0] != E or rows.shape[1] % 2:
        raise ValueError(f"W13 must be [{E}, 2 I, {H}]")
    I = rows.shape[1] // 2
    return (_weights(W13, "W13", dtype, (E,), 2 * I, H, index), _weights(W2, "W2", dtype, (E,), H, I, index), I)


def gemm_moe_ffn(X, ids, weights, W13, W2, Y, stream=None) -> None:
    """Y[t] = sum over j of weights[t, j] · W2_e (silu(G_e x_t) * (U_e x_t)), e = ids[t, j].

    W13 [E, 2 I, H] (gate rows, then up rows) and W2 [E, H, I] are tensors of X's
    type or ``W4`` stacks.  Ids outside [0, E) are skipped.  At most 64 tokens."""
    lib = _lib or _setup()
    index = _cuda(X, "X")
    dt = _type16(X, "X")
    if X.dim() != 2 or not _g._is_tensor(ids) or ids.dim() != 2:
        raise ValueError("X must be [T, H] and ids [T, k]")
    T, H = X.shape
    k = ids.shape[1]
    rows = W13.codes if isinstance(W13, W4) else W13
    if not _g._is_tensor(rows) or rows.dim() != 3:
        raise ValueError(f"W13 must be [E, 2 I, {H}]")
    E = rows.shape[0]
    w13, w2, I = _experts(W13, W2, X.dtype, H, E, index)
    _run(lib.gemm_moe_ffn, index, stream,
         (dt, X.data_ptr(), _check(ids, "ids", _torch.int32, (T, k), index),
          _check(weights, "weights", _torch.float32, (T, k), index), ctypes.byref(w13), ctypes.byref(w2),
          _check(Y, "Y", X.dtype, (T, H), index), T, H, I, E, k))


def gemm_moe_layer(X, Wr, W13, W2, Y, k: int, bias=None, scoring=MoeScoring.SOFTMAX, renormalize: bool = True,
                   stream=None) -> None:
    """A whole mixture-of-experts layer for at most 64 tokens: gemm_moe_route, then gemm_moe_ffn on its choice."""
    lib = _lib or _setup()
    index, dt, T, H, E, wr, b = _tokens(X, Wr, bias)
    w13, w2, I = _experts(W13, W2, X.dtype, H, E, index)
    _run(lib.gemm_moe_layer, index, stream,
         (dt, X.data_ptr(), wr, b, ctypes.byref(w13), ctypes.byref(w2), _check(Y, "Y", X.dtype, (T, H), index),
          T, H, I, E, k, int(scoring), 1 if renormalize else 0))
