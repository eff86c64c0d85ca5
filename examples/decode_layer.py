"""One transformer layer served in few bits: a prompt, then decode steps in one HIP graph.

The attention projections are entropy-coded 4-bit weights (lossless for their codes), the
feed-forward weights microscaled 4-bit floats, and keys and values live in a paged 4-bit
cache.  Synthetic weights, no positional encoding.

    python examples/decode_layer.py [--batch 4] [--prompt 512] [--steps 64] [--window 0]
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import entropy_coded_weight_amd as ecw  # noqa: E402


class Pages:
    """Page tables of a batch of sequences that grow: pages are taken in turn."""

    def __init__(self, batch, max_len, page_tokens):
        width = -(-max_len // page_tokens)
        self.count, self.page_tokens, self.used = batch * width, page_tokens, 0
        self.host = np.full((batch, width), -1, np.int32)
        self.table = torch.from_numpy(self.host).cuda()

    def hold(self, lens):
        """Pages for `lens` tokens of each sequence."""
        for b, n in enumerate(lens):
            for i in range(-(-n // self.page_tokens)):
                if self.host[b, i] < 0:
                    self.host[b, i], self.used = self.used, self.used + 1
        self.table.copy_(torch.from_numpy(self.host))


class Layer:
    def __init__(self, hidden=4096, heads=32, kv_heads=8, head_dim=128, inner=14336, batch=4, max_len=2048, window=0,
                 sinks=4, seed=0):
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.window, self.sinks, self.max_len = window, sinks, max_len

        def coded(rows, cols):
            codes = np.clip(np.rint(rng.laplace(0, 1.2, (rows, cols))), -8, 7).astype(np.int8)
            c = ecw.Coding(ecw.INT_CODES, rows, cols, 2, 4, 11, 128)
            return ecw.CompressedTensor(ecw.encode(c, codes, np.full(rows, 0.4 / np.sqrt(cols), np.float16)))

        def micro(rows, cols):
            g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
            return ecw.mx4_quantize((torch.randn(rows, cols, generator=g, device="cuda") / cols ** 0.5).to(torch.float16))

        self.q, self.k, self.v = (coded(n * head_dim, hidden) for n in (heads, kv_heads, kv_heads))
        self.o = coded(hidden, heads * head_dim)
        self.gate, self.up, self.down = micro(inner, hidden), micro(inner, hidden), micro(hidden, inner)
        self.pages = Pages(batch, max_len, 64)
        self.cache = ecw.KV4Cache(self.pages.count, kv_heads, head_dim)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.float16)

    def __call__(self, x, lens, starts=None):
        """x fp32 [rows, hidden], the last rows of each sequence; lens with them."""
        h = self.norm(x)
        q, k, v = (w.gemm(h).to(torch.float16).view(x.shape[0], -1, self.head_dim) for w in (self.q, self.k, self.v))
        self.cache.append(k, v, self.pages.table, lens, starts)
        a = self.cache.attend(q, self.pages.table, lens, starts, max_len=self.max_len, window=self.window,
                              sinks=self.sinks)
        x = x + self.o.gemm(a.view(x.shape[0], -1))
        h = self.norm(x)
        inner = torch.nn.functional.silu(self.gate.gemm(h)) * self.up.gemm(h)
        return x + self.down.gemm(inner.to(torch.float16))


def generate(layer, prompt, steps):
    """prompt [batch, n, hidden]: the layer over it, then `steps` times over its own last
    output, from one captured graph.  Gives the prompt's output and every step's."""
    batch, n, hidden = prompt.shape
    layer.pages.hold([n + steps] * batch)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    first = layer(prompt.reshape(batch * n, hidden), lens)
    x = first.view(batch, n, hidden)[:, -1].clone()
    outs, warm = [], torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):  # outside the capture once, over the slot that the first step fills
        layer(x, lens + 1)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        x.copy_(layer(x, lens))
    for _ in range(steps):
        graph.replay()
        outs.append(x.clone())
    return first, outs


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 4), ("prompt", 512), ("steps", 64), ("window", 0)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = Layer(batch=a.batch, max_len=a.prompt + a.steps, window=a.window)
    x = torch.randn(a.batch, a.prompt, 4096, device="cuda")
    generate(layer, x, 2)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    _, outs = generate(layer, x, a.steps)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.batch} x {a.prompt} tokens and {a.steps} steps: {begin.elapsed_time(end):.2f} ms, "
          f"output rms {outs[-1].square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
