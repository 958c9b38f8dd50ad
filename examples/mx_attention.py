"""The attention of a layer over a quantised cache: a prompt, then single tokens.

    python examples/mx_attention.py [--batch 4] [--prompt 1024] [--tokens 64]
                                    [--dim 2048] [--heads 16] [--kv-heads 4]
                                    [--head-dim 128] [--format fp8]

A step of new tokens, of every sequence of the batch, is
  a       = norm(x), in MXFP8 blocks            mx_rmsnorm
  q, k, v = a W^T                               mxfp4_matmul
  q, k    = turned by their positions           mx_rotary
  k, v    to their places in the cache's pages  mx_cache_write
  y       = attention of q over the cache       mx_attention
  out     = y W^T                               mx_quantize, mxfp4_matmul
The prompt is one step; single tokens are one captured step, replayed with
positions, slots and lengths that are written in place.  The last step's y is
compared with softmax in 64 bits over the keys and values that the cache holds.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from q4_packed_weight_amd import binding  # noqa: E402

EPS, PAGE, T = 1e-5, 16, torch.bfloat16


def quantize(w):
    codes = torch.empty(w.shape[0], w.shape[1] // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.shape[0], w.shape[1] // 32, dtype=torch.uint8, device=w.device)
    return binding.mx_quantize(w, *w.shape, "fp4", codes, scales)


class Attention:
    def __init__(self, batch, room, dim, heads, kv_heads, head_dim, fmt, device="cuda"):
        g = torch.Generator(device)
        g.manual_seed(0)
        self.dim, self.heads, self.kv_heads, self.head_dim = dim, heads, kv_heads, head_dim
        self.batch, self.fmt, self.device = batch, fmt, device
        self.width = -(-room // PAGE)
        self.pages = batch * self.width
        self.norm = torch.ones(dim, dtype=T, device=device)
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.qkv = quantize(torch.randn(self.rows, dim, generator=g, device=device) * dim ** -0.5)
        self.out = quantize(torch.randn(dim, heads * head_dim, generator=g, device=device)
                            * (heads * head_dim) ** -0.5)
        f, self.amplitude = binding.mx_rotary_frequencies(head_dim, 10000.0, "yarn", 4.0)
        self.frequencies = f.to(device)
        code = head_dim if fmt == "fp8" else head_dim // 2
        self.pool = [torch.zeros(self.pages, kv_heads, PAGE, n, dtype=torch.uint8, device=device)
                     for n in (code, head_dim // 32, code, head_dim // 32)]
        order = torch.randperm(self.pages, generator=g, device=device)
        self.table = order.view(batch, self.width).int()
        self.length = 0

    def inputs(self, n):
        """Positions, slots, starts and lengths of n more tokens of every sequence."""
        p = torch.arange(self.length, self.length + n, device=self.device)
        slots = self.table[:, p // PAGE].long() * PAGE + p % PAGE
        self.length += n
        starts = torch.arange(0, (self.batch + 1) * n, n, dtype=torch.int32, device=self.device)
        lengths = torch.full((self.batch,), self.length, dtype=torch.int32, device=self.device)
        return p.repeat(self.batch), slots.flatten(), starts, lengths

    def buffers(self, n):
        rows, hd = self.batch * n, self.heads * self.head_dim
        size = binding.mx_attention_workspace_size(rows, self.heads, self.kv_heads, self.head_dim,
                                                   self.batch, self.width, PAGE, n)
        new = lambda *s: torch.empty(*s, dtype=T, device=self.device)  # noqa: E731
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=self.device)  # noqa: E731
        return {"a": u8(rows, self.dim), "as": u8(rows, self.dim // 32), "qkv": new(rows, self.rows),
                "y": new(rows, hd), "b": u8(rows, hd), "bs": u8(rows, hd // 32),
                "out": new(rows, self.dim), "workspace": u8(size), "tokens": n}

    def step(self, x, b, positions, slots, starts, lengths):
        rows, H, HK, D = x.shape[0], self.heads, self.kv_heads, self.head_dim
        binding.mx_rmsnorm(x, None, self.norm, EPS, rows, self.dim, "fp8", None, None, b["a"], b["as"])
        binding.mxfp4_matmul(b["a"], b["as"], "fp8", *self.qkv, rows, self.dim, self.rows, b["qkv"])
        q, k, v = b["qkv"].split([H * D, HK * D, HK * D], 1)
        qk = b["qkv"][:, :(H + HK) * D]
        binding.mx_rotary(qk, positions, self.frequencies, self.amplitude, rows, H + HK, D, D, "half", qk)
        binding.mx_cache_write(k, v, slots, rows, HK, D, self.fmt, *self.pool, self.pages, PAGE)
        binding.mx_attention(q, starts, lengths, self.table, rows, H, HK, D, self.batch, self.width,
                             b["tokens"], D ** -0.5, True, 0, self.fmt, *self.pool, self.pages, PAGE,
                             b["y"], b["workspace"])
        binding.mx_quantize(b["y"], rows, H * D, "fp8", b["b"], b["bs"])
        binding.mxfp4_matmul(b["b"], b["bs"], "fp8", *self.out, rows, H * D, self.dim, b["out"])
        return b["out"]

    def reference(self, b):
        """y of the last token of each sequence, in 64 bits from what the cache holds."""
        D, G = self.head_dim, self.heads // self.kv_heads
        p = torch.arange(self.length, device=self.device)
        out = []
        for s in range(self.batch):
            slots = self.table[s, p // PAGE].long() * PAGE + p % PAGE
            k, v = (torch.empty(self.length, self.kv_heads, D, device=self.device) for _ in range(2))
            binding.mx_cache_read(slots, self.length, self.kv_heads, D, self.fmt, *self.pool, self.pages,
                                  PAGE, k, v)
            q = b["qkv"][(s + 1) * b["tokens"] - 1, :self.heads * D].double().view(self.heads, D)
            for h in range(self.heads):
                w = torch.softmax(k[:, h // G].double() @ q[h] * D ** -0.5, 0)
                out.append(w @ v[:, h // G].double())
        return torch.stack(out).view(self.batch, -1)

    def error(self, b):
        want = self.reference(b)
        got = b["y"].view(self.batch, b["tokens"], -1)[:, -1].double()
        return float((got - want).norm() / want.norm())


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=1024)
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--dim", type=int, default=2048)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--kv-heads", type=int, default=4)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--format", choices=["fp8", "fp4"], default="fp8")
    a = p.parse_args(argv)
    layer = Attention(a.batch, a.prompt + a.tokens + 1, a.dim, a.heads, a.kv_heads, a.head_dim, a.format)
    x = torch.randn(a.batch * a.prompt, a.dim, device="cuda").to(T)
    b = layer.buffers(a.prompt)
    layer.step(x, b, *layer.inputs(a.prompt))
    errors = [layer.error(b)]
    x, b = x[:a.batch].clone(), layer.buffers(1)
    held = layer.inputs(1)
    layer.step(x, b, *held)  # eager once, then captured
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        layer.step(x, b, *held)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.tokens):
        for t, new in zip(held, layer.inputs(1)):
            t.copy_(new)
        x.copy_(b["out"])
        graph.replay()
    end.record()
    errors.append(layer.error(b))
    print(f"{a.batch} sequences, {layer.length} tokens, {a.format}: "
          f"{start.elapsed_time(end) * 1e3 / a.tokens:.1f} us a token, relative error after the prompt "
          f"{errors[0]:.1e}, after the last token {errors[1]:.1e}", flush=True)
    return errors


if __name__ == "__main__":
    main()
