"""Attention over the quantised cache where its forms change over, and the
operators together: a step of a layer's attention, eager and as a graph."""
import numpy as np
import pytest
import torch

from oracle import mx
from q4_packed_weight_amd import binding
from gpu_util import DEV
from test_mx_attention_gpu import FILL, TYPES, Batch, dev, host, put, rng, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("seqs,G", [([(1, 1500)], 4), ([(80, 1500)], 2)])
def test_scales_that_jump(seqs, G, kind, fmt):
    """Runs of keys and values whose powers lie far apart: zeros, then 1, 2^24,
    2^-20, 1: references rise, fall and hold within a sequence.  Scores stay small,
    so that every key counts; the sums' errors are those of the large values."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    nk = seqs[0][1]
    run = np.array([-200, 0, 24, -20, 0])[np.minimum(np.arange(nk) // 300, 4)]
    power = np.where(run == -200, 0.0, np.exp2(np.maximum(run, -60.0)))[:, None, None]
    for i in (0, 2):
        x = b.g.standard_normal((nk, 2, 64)) * power
        b.pool.put(i, b.slots[0], *mx.quantize(x, fmt))
    b.pool.upload()
    b.scale = 2.0 ** -30
    b.check(b.run(), sample=10)


def test_an_empty_cache_gives_zeros():
    for seqs in ([(1, 700)], [(90, 700)]):
        b = Batch(seqs, 2, 2, 128, 16, "fp8", "bf16", before=0, after=0)
        b.pool.t = [torch.zeros_like(t) for t in b.pool.t]
        assert not host(b.run()).any()


@pytest.mark.parametrize("G", [2, 30])
def test_more_sequences_than_are_looked_through(G):
    """600 sequences, their tiles laid out by the longest."""
    g = rng(G)
    seqs = [(int(g.integers(0, 3)), int(n)) for n in g.integers(0, 70, 600)]
    b = Batch(seqs, 1, G, 32, 16, "fp8", "fp16")
    b.check(b.run())


def test_starts_out_of_order_stay_within_the_tensors():
    """No promise about values: nothing outside y and the workspace is written, and
    the call ends."""
    for n, nk in ((3, 5000), (40, 900)):
        b = Batch([(n, nk), (n, nk), (n, nk)], 2, 4, 64, 16, "fp8", "bf16")
        size = binding.mx_attention_workspace_size(b.T, 8, 2, 64, 3, b.width, 16, b.most)
        ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        wide = torch.full((b.T + 8, 8 * 64), FILL, dtype=torch.bfloat16, device=DEV)
        for starts in ([0, 1000000, -5, 7], [9, 3, 9, 3], [-1, -1, -1, -1], [0, b.T, 0, b.T]):
            b.starts = np.array(starts)
            b.run(y=wide[4:-4], ws=ws[:size] if size else None)
            torch.cuda.synchronize()
            assert (wide[:4] == FILL).all() and (wide[-4:] == FILL).all()
            assert (ws[size:] == 0x5A).all()


@pytest.mark.parametrize("size", [16, 24, 48, 5])
@pytest.mark.parametrize("D", [96, 128, 192, 256])
def test_chunks_by_page_size_and_head_dim(D, size):
    """Pages of whole 16 keys and others, heads that fill 64 dims and others."""
    b = Batch([(70, 500), (1, 130), (33, 33)], 2, 2, D, size, "fp8", "bf16", sharp=2.0, extra=3)
    b.check(b.run(), sample=8)
    b.table[0, 2] = -1
    b.check(b.run(window=300), window=300, hidden={0: range(2 * size, 3 * size)}, sample=8)


def test_negative_and_zero_scale():
    for seqs in ([(1, 200)], [(40, 200)]):
        b = Batch(seqs, 2, 2, 64, 16, "fp8", "bf16", sharp=2.0)
        for scale in (-0.125, 0.0):
            b.scale = scale
            b.check(b.run(), sample=10)


def test_strided_rows_on_another_stream():
    """q and y within wider rows, heads as a third dimension, a side stream."""
    b = Batch([(5, 90), (1, 40)], 2, 4, 64, 16, "fp4", "fp16")
    first = host(b.run())
    wide = torch.full((b.T, 3 * 8 * 64), 7.0, dtype=torch.float16, device=DEV)
    wide[:, 512:1024] = b.q.view(b.T, -1)
    out = torch.full((b.T, 2 * 8 * 64), FILL, dtype=torch.float16, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b.q = wide[:, 512:1024].view(b.T, 8, 64)
        b.run(y=out[:, 512:])
    torch.cuda.current_stream().wait_stream(stream)
    assert np.array_equal(host(out[:, 512:]), first)
    assert (host(out[:, :512]) == FILL).all()


class Layer:
    """norm -> projection -> rotary -> cache -> attention -> projection."""

    def __init__(self, dim, heads, kv_heads, head_dim, pages, size, fmt):
        g = torch.Generator(DEV).manual_seed(5)
        self.sizes = dim, heads, kv_heads, head_dim
        self.pages, self.size, self.fmt = pages, size, fmt
        width = (heads + 2 * kv_heads) * head_dim
        self.qkv = self.quantize(torch.randn(width, dim, generator=g, device=DEV) * dim ** -0.5)
        self.out = self.quantize(torch.randn(dim, heads * head_dim, generator=g, device=DEV) * dim ** -0.5)
        self.norm = torch.ones(dim, dtype=torch.bfloat16, device=DEV)
        f, self.amplitude = binding.mx_rotary_frequencies(head_dim, 10000.0, "linear", 2.0)
        self.frequencies = f.to(DEV)
        n = head_dim if fmt == "fp8" else head_dim // 2
        shape = pages, kv_heads, size
        self.pool = [torch.zeros(*shape, k, dtype=torch.uint8, device=DEV)
                     for k in (n, head_dim // 32) * 2]

    @staticmethod
    def quantize(w, fmt="fp4"):
        rows, cols = w.shape
        c = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV)
        s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
        return binding.mx_quantize(w, rows, cols, fmt, c, s)

    def buffers(self, T, most):
        dim, H, HK, D = self.sizes
        new = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
        n = binding.mx_attention_workspace_size(T, H, HK, D, 2, 8, self.size, most)
        return {"codes": new(T, dim, t=torch.uint8), "scales": new(T, dim // 32, t=torch.uint8),
                "qkv": new(T, (H + 2 * HK) * D), "y": new(T, H * D), "out": new(T, dim),
                "codes2": new(T, H * D, t=torch.uint8), "scales2": new(T, H * D // 32, t=torch.uint8),
                "ws": new(n, t=torch.uint8), "most": most}

    def step(self, x, b, positions, slots, starts, counts, table):
        (dim, H, HK, D), T = self.sizes, x.shape[0]
        binding.mx_rmsnorm(x, None, self.norm, 1e-5, T, dim, "fp8", None, None, b["codes"], b["scales"])
        binding.mxfp4_matmul(b["codes"], b["scales"], "fp8", *self.qkv, T, dim, (H + 2 * HK) * D, b["qkv"])
        qk = b["qkv"][:, :(H + HK) * D]
        binding.mx_rotary(qk, positions, self.frequencies, self.amplitude, T, H + HK, D, D, "half", qk)
        k, v = b["qkv"][:, H * D:(H + HK) * D], b["qkv"][:, (H + HK) * D:]
        binding.mx_cache_write(k, v, slots, T, HK, D, self.fmt, *self.pool, self.pages, self.size)
        binding.mx_attention(b["qkv"][:, :H * D], starts, counts, table, T, H, HK, D, 2, 8, b["most"],
                             D ** -0.5, True, 0, self.fmt, *self.pool, self.pages, self.size, b["y"],
                             b["ws"])
        binding.mx_quantize(b["y"], T, H * D, "fp8", b["codes2"], b["scales2"])
        binding.mxfp4_matmul(b["codes2"], b["scales2"], "fp8", *self.out, T, H * D, dim, b["out"])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_a_prompt_then_single_tokens(fmt):
    """Two sequences' prompts as one batch, then tokens one by one as a replayed
    graph, its inputs changed in place: attention equals the oracle's over the keys
    and values that the cache gives back, and those are the written rows'."""
    size, H, HK, D = 16, 8, 2, 64
    layer = Layer(256, H, HK, D, 16, size, fmt)
    g = rng(3)
    table = torch.from_numpy(g.permutation(16).reshape(2, 8).astype(np.int32)).to(DEV)
    lengths = [0, 0]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731

    def inputs(new):
        pos, slots, starts = [], [], [0]
        for s, n in enumerate(new):
            p = np.arange(lengths[s], lengths[s] + n)
            t = host(table[s]).astype(np.int64)
            pos += p.tolist()
            slots += (t[p // size] * size + p % size).tolist()
            starts.append(starts[-1] + n)
            lengths[s] += n
        return (torch.tensor(pos, device=DEV), torch.tensor(slots, device=DEV), i32(starts), i32(lengths))

    def check(b, slots, starts):
        for s in range(2):
            n = lengths[s]
            p = np.arange(n)
            all_slots = torch.from_numpy(host(table[s]).astype(np.int64)[p // size] * size + p % size).to(DEV)
            k, v = (torch.empty(n, HK, D, dtype=torch.float32, device=DEV) for _ in range(2))
            binding.mx_cache_read(all_slots, n, HK, D, fmt, *layer.pool, 16, size, k, v)
            a, e = int(starts[s]), int(starts[s + 1])
            rows = host(b["qkv"])[a:e]
            for i, want in ((0, rows[:, H * D:(H + HK) * D]), (1, rows[:, (H + HK) * D:])):
                held = mx.dequantize(*mx.quantize(want.reshape(-1, HK, D), fmt), fmt)
                assert np.array_equal(host((k, v)[i])[n - (e - a):], held)
            q, y = rows[:, :H * D].reshape(-1, H, D), host(b["y"])[a:e].reshape(-1, H, D)
            sees = np.arange(n)[None] <= np.arange(n - (e - a), n)[:, None]
            for h in range(H):
                kk, vv = host(k)[:, h // 4], host(v)[:, h // 4]
                want, mass, _, _ = mx.attention(q[:, h], kk, vv, D ** -0.5, sees)
                # half a step of bf16, a weight's rounding to fp16, fp32 sums
                assert (np.abs(y[:, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mass).all()

    pos, slots, starts, counts = inputs([37, 70])
    x = torch.randn(107, 256, device=DEV).to(torch.bfloat16)
    b = layer.buffers(107, 70)
    layer.step(x, b, pos, slots, starts, counts, table)
    check(b, slots, starts)
    b = layer.buffers(2, 1)
    x = torch.randn(2, 256, device=DEV).to(torch.bfloat16)
    held = [t.clone() for t in inputs([1, 1])]
    layer.step(x, b, held[0], held[1], held[2], held[3], table)
    check(b, held[1], held[2])
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        layer.step(x, b, held[0], held[1], held[2], held[3], table)
    for _ in range(5):
        for t, new in zip(held, inputs([1, 1])):
            t.copy_(new)
        x.normal_()
        graph.replay()
        check(b, held[1], held[2])


def test_the_example_runs():
    """Its y against 64 bits: bf16's rounding, 2^-8 at most, and no more than as much
    again for weights and sums."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mx_attention.py")
    spec = importlib.util.spec_from_file_location("mx_attention_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(["--batch", "2", "--prompt", "40", "--tokens", "5", "--dim", "256", "--heads",
                           "4", "--kv-heads", "2", "--head-dim", "64"])
    assert max(errors) <= 2.0 ** -7
