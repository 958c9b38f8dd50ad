"""The MX operators together: one step of a layer with 4-bit weights.

    python examples/mx_layer.py [--tokens 1 16] [--dim 2048] [--ffn 1024]
                                [--experts 64] [--top-k 8]

The weights are quantised to MXFP4 once.  A step is
  r, a  = norm(x + residual), a in MXFP8 blocks       mx_rmsnorm
  p     = a W^T                                       mxfp4_matmul
  r, h  = norm(p + r), h in bf16                      mx_rmsnorm
  y     = mixture of experts of h                     mxfp4_moe
and the next step's x and residual are y and r.  Steps are captured into a
graph once per number of tokens; the result is compared with the same step in
64 bits on the weights' and activations' held values, and the time printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from q4_packed_weight_amd import binding  # noqa: E402

EPS = 1e-5
T = torch.bfloat16


def quantize(w, fmt="fp4"):
    """A weight matrix [..][rows][cols] as MX codes and scales."""
    rows, cols = w.numel() // w.shape[-1], w.shape[-1]
    codes = torch.empty(*w.shape[:-1], cols // 2 if fmt == "fp4" else cols, dtype=torch.uint8,
                        device=w.device)
    scales = torch.empty(*w.shape[:-1], cols // 32, dtype=torch.uint8, device=w.device)
    binding.mx_quantize(w, rows, cols, fmt, codes, scales)
    return codes, scales


def dequantize(codes, scales, fmt="fp4"):
    cols = scales.shape[-1] * 32
    y = torch.empty(*scales.shape[:-1], cols, dtype=torch.float32, device=codes.device)
    binding.mx_dequantize(codes, scales, y.numel() // cols, cols, fmt, y)
    return y


class Layer:
    def __init__(self, dim, ffn, experts, top_k, device, seed=0):
        g = torch.Generator(device)
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.dim, self.ffn, self.experts, self.top_k = dim, ffn, experts, top_k
        self.norm1 = (1 + 0.2 * normal(dim)).to(T)
        self.norm2 = (1 + 0.2 * normal(dim)).to(T)
        self.proj = quantize(normal(dim, dim) * dim ** -0.5)
        self.router = (1.5 * dim ** -0.5 * normal(experts, dim)).to(T)
        self.bias = 0.3 * normal(experts)
        self.up = quantize(normal(experts, 2 * ffn, dim) * dim ** -0.5)
        self.down = quantize(normal(experts, dim, ffn) * ffn ** -0.5)

    def buffers(self, tokens):
        """What a step of `tokens` tokens writes."""
        dev, n = self.router.device, tokens * self.dim
        size = binding.mxfp4_moe_workspace_size(tokens, self.dim, self.ffn, self.experts,
                                                self.top_k)
        new = lambda: torch.empty(tokens, self.dim, dtype=T, device=dev)  # noqa: E731
        return {"r": new(), "p": new(), "h": new(), "y": new(),
                "codes": torch.empty(n, dtype=torch.uint8, device=dev),
                "scales": torch.empty(n // 32, dtype=torch.uint8, device=dev),
                "workspace": torch.empty(size, dtype=torch.uint8, device=dev)}

    def step(self, x, residual, b):
        n, d = x.shape[0], self.dim
        binding.mx_rmsnorm(x, residual, self.norm1, EPS, n, d, "fp8", b["r"], None, b["codes"],
                           b["scales"])
        binding.mxfp4_matmul(b["codes"], b["scales"], "fp8", *self.proj, n, d, d, b["p"])
        binding.mx_rmsnorm(b["p"], b["r"], self.norm2, EPS, n, d, None, b["r"], b["h"], None, None)
        binding.mxfp4_moe(b["h"], self.router, self.bias, *self.up, *self.down, n, d, self.ffn,
                          self.experts, self.top_k, b["y"], b["workspace"])
        return b["y"], b["r"]

    def reference(self, b):
        """y in 64 bits from the h that the step held."""
        h, f = b["h"].double(), self.ffn
        logits = h @ self.router.double().t().contiguous() + self.bias.double()
        top, chosen = torch.sort(logits, dim=-1, descending=True, stable=True)
        p, chosen = torch.softmax(top[:, :self.top_k], -1), chosen[:, :self.top_k]
        y = torch.zeros_like(h)
        for e in chosen.unique().tolist():
            t, rank = (chosen == e).nonzero(as_tuple=True)
            up = dequantize(self.up[0][e], self.up[1][e]).double()
            down = dequantize(self.down[0][e], self.down[1][e]).double()
            gu = h[t] @ up.t().contiguous()
            act = gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]
            y.index_add_(0, t, p[t, rank].unsqueeze(-1) * (act @ down.t().contiguous()))
        a = dequantize(b["codes"], b["scales"].view(-1, self.dim // 32), "fp8").double()
        return y, a @ dequantize(*self.proj).double().t().contiguous()


def run(layer, tokens, steps=200):
    """(relative error of y, of the product, microseconds a step)."""
    dev = layer.router.device
    x = torch.randn(tokens, layer.dim, device=dev).to(T)
    residual = torch.randn(tokens, layer.dim, device=dev).to(T)
    b = layer.buffers(tokens)
    layer.step(x, residual, b)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        layer.step(x, residual, b)
    torch.cuda.current_stream().wait_stream(stream)
    graph.replay()
    y, p = layer.reference(b)
    error = float((b["y"].double() - y).norm() / y.norm())
    product = float((b["p"].double() - p).norm() / p.norm())
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return error, product, start.elapsed_time(end) * 1e3 / steps


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 64])
    p.add_argument("--dim", type=int, default=2048)
    p.add_argument("--ffn", type=int, default=1024)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    a = p.parse_args(argv)
    layer = Layer(a.dim, a.ffn, a.experts, a.top_k, "cuda")
    out = []
    for tokens in a.tokens:
        error, product, us = run(layer, tokens)
        print(f"{tokens:4d} tokens: {us:8.1f} us a step, relative error of the product "
              f"{product:.1e}, of the experts' sum {error:.1e}", flush=True)
        out.append((error, product))
    return out


if __name__ == "__main__":
    main()
