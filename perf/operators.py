"""Cases that measure the 4-bit-weight and mixture-of-experts operators.

Four operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as a user calls the framework's own:

  pack    W [B, N, K] to 4-bit codes with one scale (and zero point) per group
          of consecutive k, and the values that the codes stand for
  gemm    D = A·Wᵀ with W held in 4 bits
  route   the k experts each token goes to, and their weights, from X·Wrᵀ
  layer   a whole mixture-of-experts layer for a few tokens:
          y_t = sum over the chosen e of p_te * W2_e (silu(G_e x_t) * (U_e x_t)),
          with 16-bit or 4-bit expert weights

A 4-bit weight matrix is codes [.., N, K/2] uint8 (the even k in the low four
bits), scales [.., K/group, N] in the activations' type and optional zero
points of the same shape and type: w = scale * (code - zero), zero = 8 where
there are none.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a projection of a small model, packed when it is loaded: latency
        dict(name="pack_small", op="pack", dtype="f16", B=1, N=1024, K=2048, group=64, asym=False),
        # all experts' first products of one layer at once, with zero points
        dict(name="pack_experts", op="pack", dtype="bf16", B=8, N=11000, K=4096, group=128, asym=True),
        # one token through a small projection: the smallest decode call
        dict(name="gemm_1_small", op="gemm", dtype="f16", M=1, N=1024, K=2048, group=128, asym=False),
        # one token through a large projection: bound by reading the weights
        dict(name="gemm_1", op="gemm", dtype="bf16", M=1, N=8192, K=8192, group=128, asym=False),
        # a ragged batch of sequences in decode, small groups with zero points
        dict(name="gemm_13_ragged", op="gemm", dtype="f16", M=13, N=11000, K=4128, group=32, asym=True),
        # a full decode batch
        dict(name="gemm_48", op="gemm", dtype="bf16", M=48, N=8192, K=8192, group=64, asym=False),
        # a prompt: the product is bound by arithmetic
        dict(name="gemm_512", op="gemm", dtype="bf16", M=512, N=8192, K=8192, group=128, asym=True),
        # routing of one token
        dict(name="route_1", op="route", dtype="bf16", T=1, H=2048, E=64, k=6, score="softmax", bias=False),
        # routing of a decode batch over many experts, with a selection bias
        dict(name="route_64", op="route", dtype="f16", T=64, H=8192, E=256, k=8, score="sigmoid", bias=True),
        # one token through many small experts: latency and a short weight stream
        dict(name="layer_1", op="layer", dtype="bf16", T=1, H=2048, I=1024, E=64, k=6, group=0, asym=False),
        # a small ragged batch through few large experts: a long weight stream
        dict(name="layer_16_large", op="layer", dtype="bf16", T=16, H=4096, I=8200, E=8, k=2, group=0, asym=False),
        # a decode batch through 4-bit experts, nearly all of them chosen
        dict(name="layer_64_w4", op="layer", dtype="f16", T=64, H=2048, I=1408, E=64, k=8, group=128, asym=False),
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over the logarithm of lo..hi, a multiple of `step`."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    n = min(max(int(round(n / step)) * step, -(-lo // step) * step), hi // step * step)
    return n - step if n == 3072 else n


def draw(rng):
    op = rng.choice(["pack", "gemm", "gemm", "route", "layer", "layer"])
    dtype = rng.choice(["f16", "bf16"])
    group = rng.choice([32, 64, 128])
    asym = rng.random() < 0.5
    if op == "pack":
        return dict(op=op, dtype=dtype, B=rng.randint(1, 4), N=_log(rng, 64, 16384, 8), K=_log(rng, 256, 8192, group),
                    group=group, asym=asym)
    if op == "gemm":
        M = _log(rng, 1, 64) if rng.random() < 0.75 else _log(rng, 65, 512)
        return dict(op=op, dtype=dtype, M=M, N=_log(rng, 256, 8192, 8), K=_log(rng, 256, 8192, group), group=group,
                    asym=asym)
    E = _log(rng, 8, 256)
    k = rng.randint(1, 8)
    if op == "route":
        return dict(op=op, dtype=dtype, T=_log(rng, 1, 64), H=_log(rng, 256, 8192, 8), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5)
    four = rng.random() < 0.5
    step = group if four else 8
    H = _log(rng, 256, 4096, step)
    # no more expert weights than the largest listed case holds
    most = min(8192, 8 * 4096 * 8200 // (E * H))
    I = _log(rng, 128, max(most, 256), step)
    return dict(op=op, dtype=dtype, T=_log(rng, 1, 64), H=H, I=I, E=E, k=k, group=group if four else 0,
                asym=four and asym)


# ----------------------------------------------------------------- the inputs
def _normal(gen, shape, dtype, sigma=1.0):
    # drawn in the type itself: the matrices are gigabytes
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(sigma)


def _scaled(K, dtype):
    """Scale of normal weights of variance 1/K held as codes of about +-7 (3 sigma at code 7)."""
    return 3.0 / 7.0 / math.sqrt(K)


def _w4(gen, lead, N, K, group, asym, dtype):
    """A 4-bit matrix as a checkpoint holds it: codes, scales, zero points or None."""
    codes = torch.randint(0, 256, (*lead, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    spread = torch.rand((*lead, K // group, N), generator=gen, device="cuda") + 0.5
    scales = (spread * _scaled(K, dtype)).to(dtype)
    zeros = torch.randint(6, 10, scales.shape, generator=gen, device="cuda").to(dtype) if asym else None
    return codes, scales, zeros


def _tokens(gen, T, H, dtype, Wr, k, score, bias):
    """T tokens whose choice of experts is clear: where two scores that decide it lie within the rounding of
    32-bit sums of each other there are two right answers, so such tokens are left out of a slightly longer list."""
    X = _normal(gen, (2 * T + 8, H), dtype)
    s = _scores64(X, Wr, score)
    key = (s[1] if bias is None else s[0] + bias.double()).sort(dim=1, descending=True).values
    gap = (key[:, :k] - key[:, 1:k + 1]).amin(dim=1) if key.shape[1] > k else (key[:, :-1] - key[:, 1:]).amin(dim=1)
    clear = gap > (1e-3 if bias is None else 1e-5)
    first = torch.argsort((~clear).to(torch.int8), stable=True)[:T]
    return X[first].contiguous()


def _scores64(X, Wr, score):
    logits = X.double() @ Wr.double().t()
    return (torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)), logits


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "pack":
        B, N, K, group = case["B"], case["N"], case["K"], case["group"]
        W = _normal(gen, (B, N, K), dtype, 1.0 / math.sqrt(K))
        if case["asym"]:
            W += 0.5 / math.sqrt(K)          # a mean of its own, so that a zero point is worth having
        return dict(case=case, W=W, codes=torch.empty((B, N, K // 2), dtype=torch.uint8, device="cuda"),
                    scales=torch.empty((B, K // group, N), dtype=dtype, device="cuda"),
                    zeros=torch.empty((B, K // group, N), dtype=dtype, device="cuda") if case["asym"] else None,
                    values=torch.empty((B, N, K), dtype=dtype, device="cuda"))
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        A = _normal(gen, (M, K), dtype)
        codes, scales, zeros = _w4(gen, (), N, K, case["group"], case["asym"], dtype)
        return dict(case=case, A=A, codes=codes, scales=scales, zeros=zeros,
                    D=torch.empty((M, N), dtype=dtype, device="cuda"))
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    Wr = _normal(gen, (E, H), dtype, 1.5 / math.sqrt(H))
    if op == "route":
        bias = torch.randn(E, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        X = _tokens(gen, T, H, dtype, Wr, k, case["score"], bias)
        return dict(case=case, X=X, Wr=Wr, bias=bias, ids=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                    weights=torch.empty((T, k), dtype=torch.float32, device="cuda"))
    I = case["I"]
    X = _tokens(gen, T, H, dtype, Wr, k, "softmax", None)
    s = dict(case=case, X=X, Wr=Wr, Y=torch.empty((T, H), dtype=dtype, device="cuda"))
    if case["group"]:
        s["W13"] = _w4(gen, (E,), 2 * I, H, case["group"], case["asym"], dtype)
        s["W2"] = _w4(gen, (E,), H, I, case["group"], case["asym"], dtype)
    else:
        s["W13"] = _normal(gen, (E, 2 * I, H), dtype, 1.0 / math.sqrt(H))
        s["W2"] = _normal(gen, (E, H, I), dtype, 1.0 / math.sqrt(I))
    return s


# ------------------------------------------------------------ the plain forms
def _unpack(codes):
    """uint8 codes [.., K/2] as fp32 [.., K]."""
    return torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()


def _weights32(codes, scales, zeros, group):
    """The fp32 matrix [.., N, K] that a 4-bit one stands for."""
    q = _unpack(codes).unflatten(-1, (-1, group))
    z = 8.0 if zeros is None else zeros.float().transpose(-1, -2).unsqueeze(-1)
    return ((q - z) * scales.float().transpose(-1, -2).unsqueeze(-1)).flatten(-2)


def _plain_pack(s):
    group, dtype = s["case"]["group"], s["W"].dtype
    w = s["W"].float().unflatten(-1, (-1, group))
    if s["zeros"] is None:
        amax = w.abs().amax(-1)
        scale = (amax / torch.full_like(amax, 7.0)).to(dtype)
        zero = torch.full_like(amax, 8.0)
    else:
        lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
        scale = ((hi - lo) / torch.full_like(hi, 15.0)).to(dtype)
        zero = torch.where(scale == 0, 0.0, torch.round(-lo / scale.float()).clamp(0.0, 15.0))
    f = scale.float().unsqueeze(-1)
    steps = torch.where(f == 0, 0.0, torch.round(w / f))
    values = ((steps + zero.unsqueeze(-1)).clamp(0.0, 15.0) - zero.unsqueeze(-1)) * f
    out = [scale.transpose(-1, -2).contiguous(), values.flatten(-2).to(dtype)]
    return out if s["zeros"] is None else out + [zero.transpose(-1, -2).contiguous().to(dtype)]


def _plain_route(X, Wr, k, score, bias):
    logits = X.float() @ Wr.float().t()
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    ids = torch.sort(logits if bias is None else p + bias, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    return ids.to(torch.int32), w / w.sum(1, keepdim=True)


def _pick(W, ids, group):
    """Experts `ids` (None: all) of a weight stack, in fp32."""
    if not group:
        return (W if ids is None else W[ids]).float()
    codes, scales, zeros = (None if t is None else t if ids is None else t[ids] for t in W)
    return _weights32(codes, scales, zeros, group)


def _plain_layer(s):
    case, X = s["case"], s["X"].float()
    T, I, E, k, group = case["T"], case["I"], case["E"], case["k"], case["group"]
    ids, p = _plain_route(s["X"], s["Wr"], k, "softmax", None)
    if T * k < E:          # the chosen experts' matrices, one for each (token, expert)
        flat = ids.flatten().long()
        gu = torch.bmm(_pick(s["W13"], flat, group), X.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1)
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        y = torch.bmm(_pick(s["W2"], flat, group), h.unsqueeze(-1)).squeeze(-1)
        return (y.view(T, k, -1) * p.unsqueeze(-1)).sum(1).to(s["X"].dtype)
    # every expert for every token, and the routing weights (mostly zero) on what comes out
    gates = torch.zeros((T, E), device=X.device).scatter_(1, ids.long(), p)
    gu = torch.matmul(X, _pick(s["W13"], None, group).transpose(1, 2))
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    y = torch.matmul(h * gates.t().unsqueeze(-1), _pick(s["W2"], None, group).transpose(1, 2))
    return y.sum(0).to(s["X"].dtype)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "pack":
        return _plain_pack(s)
    if case["op"] == "gemm":
        W = _weights32(s["codes"], s["scales"], s["zeros"], case["group"])
        return (s["A"].float() @ W.t()).to(s["A"].dtype)
    if case["op"] == "route":
        return list(_plain_route(s["X"], s["Wr"], case["k"], case["score"], s["bias"]))
    return _plain_layer(s)


# -------------------------------------------------------- the framework's own
def _run_own(s):
    import dense_fp16_gemm_f16_gb300 as g
    case = s["case"]
    if case["op"] == "pack":
        W4 = g.gemm_w4_quantize(s["W"], case["group"], s["codes"], s["scales"], s["zeros"])
        g.gemm_w4_dequantize(W4, s["values"])
        out = [s["scales"], s["values"]]
        return out if s["zeros"] is None else out + [s["zeros"]]
    if case["op"] == "gemm":
        g.gemm_w4_nt(s["A"], g.W4(s["codes"], s["scales"], s["zeros"], case["group"]), s["D"])
        return s["D"]
    if case["op"] == "route":
        scoring = g.MoeScoring.SOFTMAX if case["score"] == "softmax" else g.MoeScoring.SIGMOID
        g.gemm_moe_route(s["X"], s["Wr"], s["ids"], s["weights"], bias=s["bias"], scoring=scoring)
        return [s["ids"], s["weights"]]
    W13, W2 = s["W13"], s["W2"]
    if case["group"]:
        W13, W2 = g.W4(*W13, case["group"]), g.W4(*W2, case["group"])
    g.gemm_moe_layer(s["X"], s["Wr"], W13, W2, s["Y"], case["k"])
    return s["Y"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- the least that it takes
def work(case):
    op = case["op"]

    def w4(rows, K):
        return rows * K / 2 + rows * (K // case["group"]) * (4 if case["asym"] else 2)

    if op == "pack":
        n = case["B"] * case["N"] * case["K"]
        # the values come back from the codes: read again, written once
        return {"bytes": 4 * n + 2 * w4(case["B"] * case["N"], case["K"]), "flops": 8 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + 2 * M * N + w4(N, K), "flops": 2 * M * N * K}
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    if op == "route":
        return {"bytes": 2 * (T + E) * H + 8 * T * k, "flops": 2 * T * E * H}
    I = case["I"]
    # experts that T tokens with k choices each reach, when the choices are even
    reached = E * (1 - (1 - k / E) ** T) if k < E else E
    rows = w4(2 * I, H) + w4(H, I) if case["group"] else 6 * H * I
    return {"bytes": reached * rows + 2 * E * H + 4 * T * H, "flops": 6 * T * k * H * I + 2 * T * E * H}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pack":
        return _exact_pack(s)
    if case["op"] == "gemm":
        W = _exact_w4(s["codes"], s["scales"], s["zeros"], case["group"])
        return torch.einsum("mk,nk->mn", s["A"].double(), W)
    if case["op"] == "route":
        ids, p = _exact_route(s["X"], s["Wr"], case["k"], case["score"], s["bias"])
        return [ids.to(torch.int32), p]
    X, I, group = s["X"].double(), case["I"], case["group"]
    ids, p = _exact_route(s["X"], s["Wr"], case["k"], "softmax", None)
    Y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if not len(tok):
            continue
        if group:
            W13, W2 = (_exact_w4(*(None if t is None else t[e] for t in s[n]), group) for n in ("W13", "W2"))
        else:
            W13, W2 = s["W13"][e].double(), s["W2"][e].double()
        a = torch.einsum("th,ih->ti", X[tok], W13)
        gate, up = a[:, :I], a[:, I:]
        y = torch.einsum("ti,hi->th", gate / (1 + torch.exp(-gate)) * up, W2)
        Y.index_add_(0, tok, p[tok, slot, None] * y)
    return Y


def _exact_w4(codes, scales, zeros, group):
    N, half = codes.shape
    W = torch.empty((N, 2 * half), dtype=torch.float64, device=codes.device)
    W[:, 0::2] = (codes % 16).double()
    W[:, 1::2] = (codes // 16).double()
    W -= 8.0 if zeros is None else zeros.double().repeat_interleave(group, 0).t()
    W *= scales.double().repeat_interleave(group, 0).t()
    return W


def _exact_route(X, Wr, k, score, bias):
    logits = torch.einsum("th,eh->te", X.double(), Wr.double())
    if score == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p /= p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    key = p if bias is None else p + bias.double()
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    w = torch.gather(p, 1, ids)
    return ids, w / w.sum(1, keepdim=True)


def _exact_pack(s):
    """Per group: the scale is a stored 16-bit number, so it is rounded to that type; the rest is exact."""
    group, dtype, asym = s["case"]["group"], s["W"].dtype, s["zeros"] is not None
    B, N, K = s["W"].shape
    scales = torch.empty((B, K // group, N), dtype=torch.float64, device="cuda")
    zeros = torch.empty_like(scales)
    values = torch.empty((B, N, K), dtype=torch.float64, device="cuda")
    for b in range(B):
        w = s["W"][b].double().reshape(N, K // group, group)
        low = torch.minimum(w.min(-1).values, torch.zeros((), dtype=w.dtype, device="cuda"))
        high = torch.maximum(w.max(-1).values, torch.zeros((), dtype=w.dtype, device="cuda"))
        sc = ((high - low) / 15 if asym else torch.maximum(high, -low) / 7).to(dtype).double()
        safe = torch.where(sc == 0, 1.0, sc)
        z = torch.where(sc == 0, 0.0, torch.round(-low / safe)).clamp(0, 15) if asym else torch.full_like(sc, 8.0)
        q = torch.round(w / safe.unsqueeze(-1)) + z.unsqueeze(-1)
        values[b] = ((q.clamp(0, 15) - z.unsqueeze(-1)) * sc.unsqueeze(-1)).reshape(N, K)
        scales[b], zeros[b] = sc.t(), z.t()
    return [scales, values, zeros] if asym else [scales, values]
