"""Decoding steps of a small mixture-of-experts stack with 4-bit weights and, for each
request, a low-rank adapter of its own.

Every layer is a 4-bit product that adds to the stream of activations,
x <- x + rms(x) Wᵀ, and a mixture-of-experts layer on the result,
x <- x + MoE(rms(x)).  With adapters, a token's W has the product of two thin matrices
added that its request brings.  Weights are packed once; a step of all layers is
captured into a CUDA graph and replayed.  The same stack in plain PyTorch, on
the weights that the 4-bit form stands for, checks the result.

    python examples/moe_decode.py [--tokens 4] [--layers 4] [--hidden 2048] [--inner 1024] [--experts 16] [--top 4]
                                  [--adapters 3] [--rank 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp16_gemm_f16_gb300 as g  # noqa: E402


class Layer:
    def __init__(self, H, I, E, adapters, rank, dtype, gen, device):
        def draw(*shape):
            return torch.randn(*shape, generator=gen, device=device).mul_(shape[-1] ** -0.5).to(dtype)

        self.proj = g.gemm_w4_quantize(draw(H, H), group=128)
        self.router = draw(E, H)
        self.w13 = g.gemm_w4_quantize(draw(E, 2 * I, H), group=128, symmetric=False)
        self.w2 = g.gemm_w4_quantize(draw(E, H, I), group=128, symmetric=False)
        self.norms = [torch.ones(H, dtype=dtype, device=device) for _ in range(2)]
        self.lora = g.Lora(draw(adapters, rank, H), draw(adapters, H, rank), torch.full((adapters,), 0.5, device=device))


def step(layers, x, ids, top):
    z = None   # the last layer's experts' output, added to the stream by the norm that follows
    for l in layers:
        total = torch.empty_like(x)
        n = g.gemm_rmsnorm(x, l.norms[0], residual=z, total=total).Y
        y = torch.empty_like(x)
        if l.lora.A.shape[0]:
            g.gemm_lora_nt(n, l.proj, l.lora, ids, y, beta=1.0, C=total)
        else:
            g.gemm_w4_nt(n, l.proj, y, beta=1.0, C=total)
        z = torch.empty_like(y)
        g.gemm_moe_layer(g.gemm_rmsnorm(y, l.norms[1]).Y, l.router, l.w13, l.w2, z, k=top)
        x = y
    return x + z


def rms(h, dtype):
    return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)).to(dtype)


def plain_step(layers, x, ids, top):
    """The same in fp32, one expert after the other, with the library's choice of experts."""
    z = torch.zeros_like(x)
    for l in layers:
        proj = g.gemm_w4_dequantize(l.proj).float()
        w13, w2 = g.gemm_w4_dequantize(l.w13), g.gemm_w4_dequantize(l.w2)
        h = x.float() + z.float()
        n = rms(h, x.dtype).float()
        y = h.to(x.dtype).float() + n @ proj.T
        for a in range(l.lora.A.shape[0]):
            rows = (ids == a).nonzero(as_tuple=True)[0]
            y[rows] += l.lora.factors[a] * (n[rows] @ l.lora.A[a].float().T @ l.lora.B[a].float().T)
        y = y.to(x.dtype)
        n = rms(y.float(), x.dtype)
        chosen, weights = g.gemm_moe_route(n, l.router, k=top)
        z = torch.zeros(y.shape, device=x.device)
        for e in chosen.unique().tolist():
            t, j = (chosen == e).nonzero(as_tuple=True)
            gate, up = (n[t].float() @ w13[e].float().T).chunk(2, dim=-1)
            z.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().T))
        x, z = y, z.to(x.dtype)
    return x + z


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4), ("layers", 4), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("top", 4), ("steps", 50),
                          ("adapters", 3), ("rank", 16)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    torch.backends.cuda.matmul.allow_tf32 = False
    device, dtype = torch.device("cuda", 0), torch.bfloat16
    torch.cuda.set_device(device)
    gen = torch.Generator(device=device).manual_seed(0)
    layers = [Layer(a.hidden, a.inner, a.experts, a.adapters, a.rank, dtype, gen, device) for _ in range(a.layers)]
    x = torch.randn(a.tokens, a.hidden, generator=gen, device=device).to(dtype)
    # the adapter of each token's request; -1: none
    ids = torch.randint(-1, max(a.adapters, 1), (a.tokens,), generator=gen, device=device, dtype=torch.int32)

    want = plain_step(layers, x, ids, a.top)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first = step(layers, x, ids, a.top)   # allocates the stream's scratch before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(layers, x, ids, a.top)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for _ in range(5):
            graph.replay()
        begin.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
    g.gemm_f16_nt_check(device=device)
    torch.cuda.synchronize()
    if not torch.equal(first, out):
        raise SystemExit("the replayed step differs from the first one")
    # bf16 roundings of activations at about four places per layer
    error = ((out.float() - want.float()).norm() / want.float().norm()).item()
    print(f"{a.layers} layers, {a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, {a.top} per token: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us per step, relative difference from plain PyTorch {error:.1e}")
    if not error < a.layers * 2.0 ** -7:
        raise SystemExit("too far from the plain form")


if __name__ == "__main__":
    main()
