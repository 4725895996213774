"""Decoding steps of a small mixture-of-experts stack with 4-bit weights.

Every layer is a 4-bit product that adds to the stream of activations,
x <- x + rms(x) Wᵀ, and a mixture-of-experts layer on the result,
x <- x + MoE(rms(x)).  Weights are packed once; a step of all layers is
captured into a CUDA graph and replayed.  The same stack in plain PyTorch, on
the weights that the 4-bit form stands for, checks the result.

    python examples/moe_decode.py [--tokens 4] [--layers 4] [--hidden 2048] [--inner 1024] [--experts 16] [--top 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp16_gemm_f16_gb300 as g  # noqa: E402


class Layer:
    def __init__(self, H, I, E, dtype, gen, device):
        def draw(*shape):
            return torch.randn(*shape, generator=gen, device=device).mul_(shape[-1] ** -0.5).to(dtype)

        self.proj = g.gemm_w4_quantize(draw(H, H), group=128)
        self.router = draw(E, H)
        self.w13 = g.gemm_w4_quantize(draw(E, 2 * I, H), group=128, symmetric=False)
        self.w2 = g.gemm_w4_quantize(draw(E, H, I), group=128, symmetric=False)


def rms(x):
    return torch.nn.functional.rms_norm(x, (x.shape[-1],))


def step(layers, x, top):
    for l in layers:
        y = torch.empty_like(x)
        g.gemm_w4_nt(rms(x), l.proj, y, beta=1.0, C=x)
        z = torch.empty_like(y)
        g.gemm_moe_layer(rms(y), l.router, l.w13, l.w2, z, k=top)
        x = y + z
    return x


def plain_step(layers, x, top):
    """The same in fp32, one expert after the other, with the library's choice of experts."""
    for l in layers:
        proj = g.gemm_w4_dequantize(l.proj).float()
        w13, w2 = g.gemm_w4_dequantize(l.w13), g.gemm_w4_dequantize(l.w2)
        y = (x.float() + rms(x).float() @ proj.T).to(x.dtype)
        n = rms(y)
        ids, weights = g.gemm_moe_route(n, l.router, k=top)
        z = torch.zeros(y.shape, device=x.device)
        for e in ids.unique().tolist():
            t, j = (ids == e).nonzero(as_tuple=True)
            gate, up = (n[t].float() @ w13[e].float().T).chunk(2, dim=-1)
            z.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().T))
        x = y + z.to(x.dtype)
    return x


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4), ("layers", 4), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("top", 4), ("steps", 50)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    torch.backends.cuda.matmul.allow_tf32 = False
    device, dtype = torch.device("cuda", 0), torch.bfloat16
    torch.cuda.set_device(device)
    gen = torch.Generator(device=device).manual_seed(0)
    layers = [Layer(a.hidden, a.inner, a.experts, dtype, gen, device) for _ in range(a.layers)]
    x = torch.randn(a.tokens, a.hidden, generator=gen, device=device).to(dtype)

    want = plain_step(layers, x, a.top)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first = step(layers, x, a.top)   # allocates the stream's scratch before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(layers, x, a.top)
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
