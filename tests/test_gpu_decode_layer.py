"""The layer example end to end: every output against the same layer in float64 over the
values that its coded weights and cache stand for.

Tolerance: the layer rounds to fp16 after each norm, projection, attention and gate (half
a step, 2^-11, each), and a step's input is the last step's output.  Rounded keys and
values may fall on the other side of a 4-bit border than the reference's, so the
reference takes them from the cache itself.  Eight roundings in a row of magnitude 2^-11
on sums whose terms cancel by up to a factor of about 8 give 2^-5 of the output's rms."""
import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from examples import decode_layer as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _reference(layer, x, b, total, n):
    """Rows x [n, hidden] float64, the last n of sequence b's `total` tokens."""
    w = {k: getattr(layer, k).dequantize(torch.float16).double() if k in "qkvo" else
         getattr(layer, k).dequantize(torch.float32).double() for k in ("q", "o", "gate", "up", "down")}
    norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    h = norm(x)
    q = (h @ w["q"].t()).view(n, layer.kv_heads, -1, layer.head_dim)
    k, v = layer.cache.read(layer.pages.table[b:b + 1], torch.tensor([total], dtype=torch.int32, device="cuda"), total,
                            dtype=torch.float32)
    s = torch.einsum("nhgd,thd->nhgt", q, k.double()) * layer.head_dim ** -0.5
    at = torch.arange(total - n, total, device="cuda")[:, None]
    t = torch.arange(total, device="cuda")
    seen = t <= at
    if layer.window:
        seen &= (t > at - layer.window) | (t < layer.sinks)
    p = torch.softmax(s.masked_fill(~seen[:, None, None], -float("inf")), -1)
    x = x + torch.einsum("nhgt,thd->nhgd", p, v.double()).reshape(n, -1) @ w["o"].t()
    h = norm(x)
    return x + (torch.nn.functional.silu(h @ w["gate"].t()) * (h @ w["up"].t())) @ w["down"].t()


@pytest.mark.parametrize("batch,window", [(1, 0), (3, 0), (6, 40)])
def test_prompt_and_steps(batch, window):
    print("[gpu] decode layer", batch, window, flush=True)
    layer = D.Layer(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=768, batch=batch, max_len=160, window=window,
                    seed=3)
    x = torch.randn(batch, 130, 512, generator=torch.Generator().manual_seed(1)).cuda()
    first, outs = D.generate(layer, x, 5)
    torch.cuda.synchronize()
    for b in range(batch):
        want = _reference(layer, x[b].double(), b, 130, 130)
        got = first.view(batch, 130, 512)[b].double()
        assert float((got - want).abs().max()) <= 2.0 ** -5 * float(want.square().mean().sqrt())
        before = got[-1:]
        for i, o in enumerate(outs):
            want = _reference(layer, before, b, 131 + i, 1)
            assert float((o[b].double() - want).abs().max()) <= 2.0 ** -5 * float(want.square().mean().sqrt())
            before = o[b:b + 1].double()
    assert np.isfinite(float(outs[-1].sum()))
    assert isinstance(layer.gate, ecw.MX4Tensor)


def _step_of_four_bits(x):
    """How far the 4-bit value of a number may be from it, where the number itself is known
    to 2^-9 of its block's largest: the half step of its magnitude (2 units at 8, which becomes
    6), for either scale if the largest lies that close to a power of two."""
    blocks = np.abs(x.reshape(*x.shape[:-1], -1, 32))
    top = blocks.max(-1, keepdims=True)
    most = np.zeros_like(blocks)
    for near in (1 - 2.0 ** -9, 1 + 2.0 ** -9):
        s = np.exp2(np.floor(np.log2(top * near)) - 2)
        u = (blocks + 2.0 ** -9 * top) / s
        most = np.maximum(most, s * np.where(u > 6, np.maximum(u - 6, 1), np.where(u > 4, 1, np.where(u > 2, 0.5, 0.25))))
    return (most + 2.0 ** -9 * top).reshape(x.shape)


@pytest.mark.parametrize("batch,window", [(1, 0), (3, 40), (6, 0)])
def test_cache_holds_the_layers_own_keys_and_values(batch, window):
    """What the prompt and every replay of the graph append are the k and v projections of
    their own input, at their own place: the projections in float64, within 4 bits of them.
    (The projections' own error, fp32 sums and an fp16 rounding of 2^-11, stays under 2^-9 of
    a block's largest.)"""
    print("[gpu] decode layer cache", batch, window, flush=True)
    layer = D.Layer(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=768, batch=batch, max_len=160, window=window,
                    seed=5)
    x = torch.randn(batch, 130, 512, generator=torch.Generator().manual_seed(2)).cuda()
    first, outs = D.generate(layer, x, 5)
    torch.cuda.synchronize()
    inputs = torch.cat([x, first.view(batch, 130, 512)[:, -1:], *(o[:, None] for o in outs[:-1])], 1)
    lens = torch.full((batch,), 135, dtype=torch.int32, device="cuda")
    held = layer.cache.read(layer.pages.table, lens, batch * 135, dtype=torch.float32)
    h = layer.norm(inputs.reshape(batch * 135, 512)).double()
    for got, w in zip(held, (layer.k, layer.v)):
        want = (h @ w.dequantize(torch.float16).double().t()).view(-1, 2, 64).cpu().numpy()
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= _step_of_four_bits(want)).all(), f"worst {(err / _step_of_four_bits(want)).max()}"
