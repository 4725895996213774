"""Cases that measure the normalisation, the row-scaled 8-bit product and the low-rank adapters.

Each in a plain form (elementary torch operations in 32 bits, rounded once at
the end) and as a user calls the framework's own:

  norm   h = x + r, y = h / sqrt(mean(h^2) + eps) * w: y in 16 bits, y in 8 bits
         with a scale per row (max|y| / the type's largest number), h in 16 bits
  prod   D = sm[m] * sn[n] * (A Bt) + bias[n] with A and B in 8 bits, D in bf16
  lora   D[m] = X[m] Wt + c_a (X[m] A_at) B_at + C[m], a = ids[m] (-1: none), with
         W in 16 bits or in 4
  block  the three together: a normalised row in 16 and 8 bits, the adapters'
         part from the first, the product of the second with it as the addend

A 4-bit W is codes [N, K/2] uint8 (the even k in the low four bits) and scales
[K/group, N] in the activations' type: w = scale * (code - 8).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a small model between two products: latency
        dict(name="norm_1", op="norm", dtype="bf16", T=1, H=2048, residual=True, y16=True, y8=""),
        # a ragged decode batch whose rows go to a 16-bit router and an 8-bit product
        dict(name="norm_37_both", op="norm", dtype="f16", T=37, H=5128, residual=True, y16=True, y8="e4m3"),
        # a prompt's tokens for 8-bit products: bound by the bytes
        dict(name="norm_4096_8bit", op="norm", dtype="bf16", T=4096, H=8192, residual=True, y16=False, y8="e4m3"),
        # a few tokens through a small 8-bit projection
        dict(name="prod_3", op="prod", fmt="e4m3", M=3, N=2048, K=2048, bias=False),
        # a decode batch through a large projection: bound by the weights' bytes
        dict(name="prod_48", op="prod", fmt="e4m3", M=48, N=8192, K=8192, bias=False),
        # a ragged prompt: bound by the 8-bit tensor rate
        dict(name="prod_4000", op="prod", fmt="e5m2", M=4000, N=8200, K=8192, bias=True),
        # one token of one adapter through a small projection: latency
        dict(name="lora_1", op="lora", dtype="f16", M=1, N=1024, K=2048, R=8, count=4, runs=False, group=0, add=False),
        # a decode batch of requests with adapters of their own, residual added in the product
        dict(name="lora_16", op="lora", dtype="bf16", M=16, N=8192, K=8192, R=16, count=32, runs=False, group=0, add=True),
        # a larger decode batch, high ranks, beside 4-bit weights
        dict(name="lora_61_w4", op="lora", dtype="bf16", M=61, N=8192, K=4096, R=64, count=48, runs=False, group=128,
             add=False),
        # a very large decode batch: adapters in any order, ragged sizes
        dict(name="lora_250", op="lora", dtype="f16", M=250, N=5000, K=4104, R=32, count=64, runs=False, group=0, add=False),
        # prompts of a few requests one behind the other
        dict(name="lora_4096_runs", op="lora", dtype="bf16", M=4096, N=8192, K=8192, R=16, count=8, runs=True, group=0,
             add=False),
        # a decode batch through norm, adapters and the 8-bit product
        dict(name="block_32", op="block", dtype="bf16", fmt="e4m3", M=32, N=8192, K=8192, R=16, count=16, runs=False),
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over the logarithm of lo..hi, a multiple of `step`."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(int(round(n / step)) * step, -(-lo // step) * step), hi // step * step)


def _rows(rng):
    """Rows of a product: mostly decode batches, some prompts."""
    return _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 65, 4096)


def draw(rng):
    op = rng.choice(["norm", "norm", "prod", "lora", "lora", "lora", "block"])
    if op == "norm":
        H = _log(rng, 64, 16384, 8)
        y8 = rng.choice(["", "e4m3", "e4m3", "e5m2"])
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), T=_log(rng, 1, min(8192, 4096 * 8192 // H)), H=H,
                    residual=rng.random() < 0.7, y16=not y8 or rng.random() < 0.5, y8=y8)
    if op == "prod":
        return dict(op=op, fmt=rng.choice(["e4m3", "e5m2"]), M=min(4000, _rows(rng)), N=_log(rng, 256, 8192, 8),
                    K=_log(rng, 256, 8192, 16), bias=rng.random() < 0.5)
    M, R, count = _rows(rng), rng.choice([8, 16, 24, 32, 64, 128]), _log(rng, 1, 64)
    runs = M > 64 and rng.random() < 0.6
    if op == "block":
        return dict(op=op, dtype="bf16", fmt=rng.choice(["e4m3", "e5m2"]), M=min(M, 2048), N=_log(rng, 256, 8192, 8),
                    K=_log(rng, 256, 8192, 16), R=R, count=count, runs=runs)
    group = rng.choice([0, 0, 32, 64, 128])
    return dict(op=op, dtype=rng.choice(["f16", "bf16"]), M=M, N=_log(rng, 256, 8192, 8),
                K=_log(rng, 256, 8192, group or 8), R=R, count=count, runs=runs, group=group, add=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs
def _normal(gen, shape, dtype, sigma=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(sigma)


def _uniform(gen, shape, lo, hi):
    return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo


def _eight(gen, rows, K, fmt):
    """Rows in 8 bits as a row-wise quantisation leaves them (normal values, the largest near the type's), and their scales."""
    kind, top = FORMATS[fmt]
    codes = _normal(gen, (rows, K), torch.float32, top / 5.0).clamp_(-top, top).to(kind)
    return codes, _uniform(gen, (rows,), 0.5, 1.5) * (5.0 / top)


def _adapters(gen, case, dtype):
    """Adapters A [count, R, K], B [count, N, R] and factors; the adapter of each row, -1 for about one in ten."""
    count, R, K, N, M = case["count"], case["R"], case["K"], case["N"], case["M"]
    A = _normal(gen, (count, R, K), dtype, K ** -0.5)
    B = _normal(gen, (count, N, R), dtype, R ** -0.5)
    factors = _uniform(gen, (count,), 0.1, 0.5)
    ids = torch.randint(0, count, (M,), generator=gen, device="cuda", dtype=torch.int32)
    ids[torch.rand(M, generator=gen, device="cuda") < 0.1] = -1
    if case["runs"]:
        # prompts of uneven length one behind the other
        starts = torch.rand(M, generator=gen, device="cuda") < 6.0 / M
        starts[0] = True
        ids = ids[starts.long().cumsum(0) - 1]
    return A, B, factors, ids.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "prod":
        A, sm = _eight(gen, case["M"], case["K"], case["fmt"])
        B, sn = _eight(gen, case["N"], case["K"], case["fmt"])
        sn *= case["K"] ** -0.5
        bias = _normal(gen, (case["N"],), torch.bfloat16) if case["bias"] else None
        return dict(case=case, A=A, sm=sm, B=B, sn=sn, bias=bias,
                    D=torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda"))
    dtype = DTYPES[case["dtype"]]
    if op in ("norm", "block"):
        T, H = (case["T"], case["H"]) if op == "norm" else (case["M"], case["K"])
        # activations with a few channels far above the others
        loud = torch.where(torch.rand(H, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
        s = dict(case=case, X=(_normal(gen, (T, H), torch.float32) * loud).to(dtype),
                 w=_uniform(gen, (H,), 0.5, 1.5).to(dtype))
        s["r"] = _normal(gen, (T, H), dtype, 2.0) if op == "block" or case["residual"] else None
        s["total"] = None if s["r"] is None else torch.empty((T, H), dtype=dtype, device="cuda")
        s["Y"] = torch.empty((T, H), dtype=dtype, device="cuda") if op == "block" or case["y16"] else None
        kind = "e4m3" if op == "norm" and not case["y8"] else case["fmt"] if op == "block" else case["y8"]
        eight = op == "block" or case["y8"]
        s["Y8"] = torch.empty((T, H), dtype=FORMATS[kind][0], device="cuda") if eight else None
        s["scales"] = torch.empty((T,), dtype=torch.float32, device="cuda") if eight else None
        if op == "norm":
            return s
        s["W8"], s["sn"] = _eight(gen, case["N"], H, case["fmt"])
        s["sn"] *= H ** -0.5
        s["A"], s["B"], s["factors"], s["ids"] = _adapters(gen, case, dtype)
        s["U"], s["D"] = (torch.empty((T, case["N"]), dtype=dtype, device="cuda") for _ in range(2))
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s = dict(case=case, X=_normal(gen, (M, K), dtype), D=torch.empty((M, N), dtype=dtype, device="cuda"))
    if case["group"]:
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["wscales"] = (_uniform(gen, (K // case["group"], N), 0.5, 1.5) * (0.2 * K ** -0.5)).to(dtype)
    else:
        s["W"] = _normal(gen, (N, K), dtype, K ** -0.5)
    s["A"], s["B"], s["factors"], s["ids"] = _adapters(gen, case, dtype)
    s["C"] = _normal(gen, (M, N), dtype) if case["add"] else None
    return s


# ------------------------------------------------------------ the plain forms
def _plain_norm(s):
    """(y in 32 bits, the outputs that are asked for)."""
    h = s["X"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    out = {}
    if s["Y"] is not None:
        out["y"] = y.to(s["X"].dtype)
    if s["Y8"] is not None:
        kind = s["Y8"].dtype
        top = FORMATS["e5m2" if kind == torch.float8_e5m2 else "e4m3"][1]
        amax = y.abs().amax(1)
        scales = amax / torch.full_like(amax, top)
        out["y8"] = (y / scales[:, None]).clamp(-top, top).to(kind)
        out["scales"] = scales
    if s["total"] is not None:
        out["total"] = h.to(s["X"].dtype)
    return out


def _plain_adapters(X, A, B, factors, ids):
    """c_a (x A_at) B_at in 32 bits: every adapter's low-rank rows, those of other adapters taken out, times all B."""
    count, R, K = A.shape
    low = (X.float() @ A.float().view(count * R, K).t()).view(-1, count, R)
    mine = ids[:, None] == torch.arange(count, device=ids.device)
    low = low * torch.where(mine, factors, 0.0)[:, :, None]
    return low.flatten(1) @ B.float().transpose(1, 2).reshape(count * R, -1)


def _plain_prod(A, sm, B, sn):
    return (A.float() @ B.float().t()) * sm[:, None] * sn


def _weights32(s):
    if not s["case"]["group"]:
        return s["W"].float()
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).flatten(-2).float().unflatten(-1, (-1, s["case"]["group"]))
    return ((q - 8.0) * s["wscales"].float().t().unsqueeze(-1)).flatten(-2)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "prod":
        d = _plain_prod(s["A"], s["sm"], s["B"], s["sn"])
        return (d if s["bias"] is None else d + s["bias"].float()).to(torch.bfloat16)
    if op == "block":
        n = _plain_norm(s)
        d = _plain_prod(n["y8"], n["scales"], s["W8"], s["sn"])
        d = d + _plain_adapters(n["y"], s["A"], s["B"], s["factors"], s["ids"])
        return {"d": d.to(s["X"].dtype), "total": n["total"]}
    d = s["X"].float() @ _weights32(s).t() + _plain_adapters(s["X"], s["A"], s["B"], s["factors"], s["ids"])
    return (d if s["C"] is None else d + s["C"].float()).to(s["X"].dtype)


# -------------------------------------------------------- the framework's own
def _own_norm(g, s):
    g.gemm_rmsnorm(s["X"], s["w"], residual=s["r"], eps=EPS, Y=s["Y"], Y8=s["Y8"], scales=s["scales"], total=s["total"])
    return {k: s[n] for k, n in (("y", "Y"), ("y8", "Y8"), ("scales", "scales"), ("total", "total")) if s[n] is not None}


def _run_own(s):
    import dense_fp16_gemm_f16_gb300 as g
    case = s["case"]
    if case["op"] == "norm":
        return _own_norm(g, s)
    if case["op"] == "prod":
        g.gemm_nt_ex(s["A"], s["B"], s["D"], scale_m=s["sm"], scale_n=s["sn"], bias=s["bias"])
        return s["D"]
    lora = g.Lora(s["A"], s["B"], s["factors"])
    if case["op"] == "block":
        _own_norm(g, s)
        g.gemm_lora_delta(s["Y"], lora, s["ids"], s["U"])
        g.gemm_nt_ex(s["Y8"], s["W8"], s["D"], scale_m=s["scales"], scale_n=s["sn"], beta=1.0, C=s["U"])
        return {"d": s["D"], "total": s["total"]}
    W = g.W4(s["codes"], s["wscales"], None, case["group"]) if case["group"] else s["W"]
    if s["C"] is None:
        g.gemm_lora_nt(s["X"], W, lora, s["ids"], s["D"])
    else:
        g.gemm_lora_nt(s["X"], W, lora, s["ids"], s["D"], beta=1.0, C=s["C"])
    return s["D"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- the least that it takes
def work(case):
    op = case["op"]

    def norm(T, H, residual, y16, y8):
        return T * H * (2 + 4 * residual + 2 * y16 + y8) + 2 * H, T * H * (6 + 3 * y8)

    def adapters(M, N, K, R, count, runs):
        """Bytes of the adapters that the rows reach, when the choices are even, and the flops of their rows."""
        picks = min(M, 7) if runs else 0.9 * M
        return count * (1 - (1 - 1 / count) ** picks) * 2 * R * (K + N), 0.9 * M * 2 * R * (K + N)

    if op == "norm":
        b, f = norm(case["T"], case["H"], case["residual"], case["y16"], bool(case["y8"]))
        return {"bytes": b, "flops": f}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "prod":
        return {"bytes": (M + N) * K + 2 * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    low, low_flops = adapters(M, N, K, case["R"], case["count"], case["runs"])
    if op == "block":
        # y in both forms stays on the way: read and written by no more than one call each
        b, f = norm(M, K, True, False, False)
        return {"bytes": b + low + N * K + 2 * M * N, "flops": f + low_flops + 2 * M * N * K}
    weights = N * K / 2 + 2 * N * (K // case["group"]) if case["group"] else 2 * N * K
    return {"bytes": weights + low + 2 * M * K + (4 if case["add"] else 2) * M * N, "flops": 2 * M * N * K + low_flops}


# ------------------------------------------------------------- in 64 bits
def _round8(v, fmt):
    """float64 numbers rounded to the nearest of an 8-bit type, ties to even, beyond the largest to the largest."""
    fraction, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    exponent = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(torch.clamp(exponent, min=lowest) - fraction)
    top = FORMATS[fmt][1]
    return torch.clamp(torch.round(v / step) * step, -top, top)


def _exact_norm(s, fmt):
    h = s["X"].double()
    if s["r"] is not None:
        h += s["r"].double()
    rms = torch.sqrt(torch.einsum("th,th->t", h, h) / h.shape[1] + EPS)
    y = torch.einsum("th,t,h->th", h, 1 / rms, s["w"].double())
    out = {"y64": y, "total": h, "y": y}
    if fmt:
        # a scale is a stored 32-bit number
        out["scales"] = (torch.maximum(y.amax(1), -y.amin(1)) / FORMATS[fmt][1]).float().double()
        out["y8"] = _round8(y / out["scales"][:, None], fmt)
    return out


def _exact_adapters(X, s):
    out = torch.zeros((X.shape[0], s["B"].shape[1]), dtype=torch.float64, device="cuda")
    for a in range(s["A"].shape[0]):
        rows = (s["ids"] == a).nonzero(as_tuple=True)[0]
        if len(rows):
            low = torch.einsum("tk,rk->tr", X[rows], s["A"][a].double()) * s["factors"][a].double()
            out[rows] = torch.einsum("tr,nr->tn", low, s["B"][a].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        got = _exact_norm(s, case["y8"])
        keep = (["y"] if case["y16"] else []) + (["y8", "scales"] if case["y8"] else []) + (["total"] if case["residual"] else [])
        return {k: got[k] for k in keep}
    if op == "prod":
        d = torch.einsum("mk,nk->mn", s["A"].double(), s["B"].double()) * s["sm"].double()[:, None] * s["sn"].double()[None]
        return d if s["bias"] is None else d + s["bias"].double()[None]
    if op == "block":
        n = _exact_norm(s, case["fmt"])
        d = torch.einsum("mk,nk->mn", n["y8"] * n["scales"][:, None], s["W8"].double() * s["sn"].double()[:, None])
        # the 16-bit rows that the adapters read are stored numbers
        return {"d": d + _exact_adapters(n["y64"].to(s["X"].dtype).double(), s), "total": n["total"]}
    if case["group"]:
        N, half = s["codes"].shape
        W = torch.empty((N, 2 * half), dtype=torch.float64, device="cuda")
        W[:, 0::2], W[:, 1::2] = (s["codes"] % 16).double(), (s["codes"] // 16).double()
        W = (W - 8.0) * s["wscales"].double().repeat_interleave(case["group"], 0).t()
    else:
        W = s["W"].double()
    d = torch.einsum("mk,nk->mn", s["X"].double(), W) + _exact_adapters(s["X"].double(), s)
    return d if s["C"] is None else d + s["C"].double()
