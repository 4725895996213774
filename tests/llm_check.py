"""Plain 64-bit forms of the 4-bit-weight and mixture-of-experts operators, and
the bounds that the GPU results are held to.

Bounds, per output element, fixed from the arithmetic before any run:
  u |ref|          the one rounding of the output (u = half an ulp of a number just
                   above a power of two: 2^-11 for fp16's 11 significant bits, 2^-8
                   for bf16's 8), taken 1 % wider for the sums' own error
  2^-22 S          fp32 sums, S = sum of the magnitudes that enter them.  A
                   4-bit code may enter as code + 128 with the offset taken out
                   afterwards, so S counts |x| |s| (code + |z| + 128)
  2^-25            half the spacing of fp16's subnormal numbers
"""
from __future__ import annotations

import torch

import dense_fp16_gemm_f16_gb300 as g

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E32 = 2.0 ** -22
FLOOR = 2.0 ** -25


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double()


def w64(W):
    """(exact weights, magnitudes that enter the sums) of a 16-bit tensor or a W4, in float64."""
    if not isinstance(W, g.W4):
        w = W.double()
        return w, w.abs()
    q = unpack(W.codes)
    s = W.scales.double().transpose(-1, -2).repeat_interleave(W.group, -1)
    z = 8.0 if W.zeros is None else W.zeros.double().transpose(-1, -2).repeat_interleave(W.group, -1)
    return (q - z) * s, (q + (z if W.zeros is None else z.abs()) + 128.0) * s.abs()


def random_w4(gen, lead, N, K, group, asym, dtype, device="cuda"):
    codes = torch.randint(0, 256, (*lead, N, K // 2), generator=gen, dtype=torch.uint8)
    scales = ((torch.rand((*lead, K // group, N), generator=gen) + 0.5) * 0.4 / K ** 0.5).to(dtype)
    # the sign of a scale is free, and zero points need not be whole
    scales = torch.where(torch.rand(scales.shape, generator=gen) < 0.1, -scales, scales)
    zeros = (torch.randint(0, 31, scales.shape, generator=gen) / 2).to(dtype) if asym else None
    return g.W4(codes.to(device), scales.to(device), None if zeros is None else zeros.to(device), group)


def check(got, ref, tol, what):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst "
                                 f"{float(((got - ref).abs() / tol)[bad].max())} times the bound; first at "
                                 f"{bad.nonzero()[0].tolist()}")


def quantize64(W, group, asym):
    """(codes, scales, zeros or None) by the definition; 64-bit but for the stored 16-bit scale."""
    dtype = W.dtype
    w = W.double().unflatten(-1, (-1, group))
    lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
    s = ((hi - lo).float() / torch.full_like(hi, 15, dtype=torch.float32) if asym else
         torch.maximum(hi, -lo).float() / torch.full_like(hi, 7, dtype=torch.float32)).to(dtype)
    f = s.double()
    safe = torch.where(f == 0, 1.0, f)
    z = torch.where(f == 0, 0.0, torch.round(-lo / safe).clamp(0, 15)) if asym else torch.full_like(f, 8.0)
    q = torch.where((f == 0)[..., None], 0.0, torch.round(w / safe[..., None])) + z[..., None]
    q = q.clamp(0, 15).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), s.transpose(-1, -2), z.to(dtype).transpose(-1, -2) if asym else None


def route64(X, Wr, k, bias=None, scoring=0, renormalize=True):
    logits = X.double() @ Wr.double().t()
    p = torch.softmax(logits, 1) if scoring == 0 else torch.sigmoid(logits)
    key = logits if bias is None else p + bias.double()
    key = torch.where(torch.isnan(key), -torch.inf, key)
    ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
    out = torch.gather(key, 1, ids) == -torch.inf
    w = torch.gather(p, 1, ids).masked_fill(out, 0.0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, w, w / total)
    return ids.masked_fill(out, -1).to(torch.int32), w


def ffn64(X, ids, weights, W13, W2):
    """(Y, bound) in 64 bits.  The bound follows h through both products: fp32 sums
    (2^-22 of their magnitudes), exp and division in fp32 (2^-20 of h), and h kept as a
    sum of two numbers of X's type (2^-16 of h covers both types, 2^-24 fp16's subnormals)."""
    T, H = X.shape
    E = (W13.codes if isinstance(W13, g.W4) else W13).shape[0]
    Y = torch.zeros((T, H), dtype=torch.float64, device=X.device)
    err = torch.zeros_like(Y)
    for e in range(E):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if not len(tok):
            continue
        one = [g.W4(w.codes[e], w.scales[e], None if w.zeros is None else w.zeros[e], w.group)
               if isinstance(w, g.W4) else w[e] for w in (W13, W2)]
        (a, am), (b, bm) = w64(one[0]), w64(one[1])
        I = b.shape[1]
        x = X[tok].double()
        gu, mag = x @ a.t(), x.abs() @ am.t()
        gate, up = gu[:, :I], gu[:, I:]
        sig = torch.sigmoid(gate)
        h = gate * sig * up
        # |d silu / d gate| <= 1.1
        eh = E32 * (1.1 * mag[:, :I] * up.abs() + mag[:, I:] * (gate * sig).abs()) + 2.0 ** -16 * h.abs() + 2.0 ** -24
        w = weights[tok, slot, None].double()
        Y.index_add_(0, tok, w * (h @ b.t()))
        err.index_add_(0, tok, w.abs() * (eh @ b.abs().t() + E32 * (h.abs() @ bm.t())))
    return Y, 1.01 * U[X.dtype] * Y.abs() + err + FLOOR
