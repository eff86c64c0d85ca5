"""The layer example with its feed-forward in 8 bits and rotary positions: norm, products,
gate, rotation, cache and attention as they follow each other, eagerly and in one graph.

Tolerance: everything up to the feed-forward rounds to fp16 (2^-11) as in the 4-bit example,
2^-5 of the output's rms together.  In the feed-forward the reference rounds to 8 bits too,
but its inputs differ by about 2^-9 relative, which puts under 2^-4 of the numbers (twice
2^-9 over a step of 2^-4 at least) on the other side of a border, a step of 2^-3 at most
away: 2^-5 of the 2-norm for each of two roundings, and the gate doubles the first at most.
bf16 between the products adds 2^-9.  So 2^-3 of the feed-forward's own 2-norm."""
import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from examples import decode_layer as D
from tests import fp8_ref as R
from tests.test_gpu_decode_layer import _step_of_four_bits

pytestmark = pytest.mark.gpu
BASE = 500000.0


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _norm(t):
    return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)


def _rotated(x, positions):
    """x [rows, heads, dim] float64 at positions [rows]."""
    half = x.shape[-1] // 2
    angle = positions.double()[:, None] * BASE ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    return torch.from_numpy(R.rotate(x.cpu().numpy(), torch.cos(angle).cpu().numpy(), torch.sin(angle).cpu().numpy(), 2 * half, False)).cuda()


def _rounded(x):
    return torch.from_numpy(R.rounded(x.cpu().numpy())).cuda()


def _reference(layer, x, b, total, n):
    """Rows x [n, hidden] float64, the last n of sequence b's `total` tokens: what goes into the
    feed-forward, and what it adds."""
    w = {k: getattr(layer, k).dequantize(torch.float16).double() for k in "qo"}
    positions = torch.arange(total - n, total, device="cuda")
    q = _rotated((_norm(x) @ w["q"].t()).view(n, -1, layer.head_dim), positions).view(n, layer.kv_heads, -1, layer.head_dim)
    k, v = layer.cache.read(layer.pages.table[b:b + 1], torch.tensor([total], dtype=torch.int32, device="cuda"), total,
                            dtype=torch.float32)
    s = torch.einsum("nhgd,thd->nhgt", q, k.double()) * layer.head_dim ** -0.5
    p = torch.softmax(s.masked_fill(~(torch.arange(total, device="cuda") <= positions[:, None])[:, None, None], -float("inf")), -1)
    x = x + torch.einsum("nhgt,thd->nhgd", p, v.double()).reshape(n, -1) @ w["o"].t()
    both = _rounded(_norm(x)) @ layer.gate_up.dequantize(torch.float32).double().t()
    gate, up = both[:, :layer.inner], both[:, layer.inner:]
    return x, _rounded(torch.nn.functional.silu(gate) * up) @ layer.down.dequantize(torch.float32).double().t()


def _near(got, middle, added):
    err = (got - middle - added).norm()
    return err <= 2.0 ** -3 * added.norm() + 2.0 ** -5 * middle.norm()


@pytest.mark.parametrize("batch", [1, 3, 20])
def test_prompt_and_steps(batch):
    print("[gpu] 8-bit decode layer", batch, flush=True)
    layer = D.Layer(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=768, batch=batch, max_len=160, seed=3, feed="fp8",
                    rotary=BASE)
    x = torch.randn(batch, 130, 512, generator=torch.Generator().manual_seed(1)).cuda()
    first, outs = D.generate(layer, x, 5)
    torch.cuda.synchronize()
    for b in range(min(batch, 3)):
        got = first.view(batch, 130, 512)[b].double()
        assert _near(got, *_reference(layer, x[b].double(), b, 130, 130))
        before = got[-1:]
        for i, o in enumerate(outs):
            assert _near(o[b:b + 1].double(), *_reference(layer, before, b, 131 + i, 1))
            before = o[b:b + 1].double()
    assert np.isfinite(float(outs[-1].sum()))
    assert isinstance(layer.gate_up, ecw.FP8Tensor)


def test_cache_holds_rotated_keys():
    """What the prompt and every replay of the graph append are the k projections of their own
    input, turned by their own place; values are not turned."""
    batch = 3
    layer = D.Layer(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=768, batch=batch, max_len=160, seed=5, feed="fp8",
                    rotary=BASE)
    x = torch.randn(batch, 130, 512, generator=torch.Generator().manual_seed(2)).cuda()
    first, outs = D.generate(layer, x, 5)
    torch.cuda.synchronize()
    inputs = torch.cat([x, first.view(batch, 130, 512)[:, -1:], *(o[:, None] for o in outs[:-1])], 1)
    lens = torch.full((batch,), 135, dtype=torch.int32, device="cuda")
    held = layer.cache.read(layer.pages.table, lens, batch * 135, dtype=torch.float32)
    h = ecw.rms_norm(inputs.reshape(batch * 135, 512), out_dtype=torch.float16).double()
    for got, w, turn in zip(held, (layer.k, layer.v), (True, False)):
        want = (h @ w.dequantize(torch.float16).double().t()).view(-1, 2, 64)
        if turn:
            want = _rotated(want, torch.arange(135, device="cuda").repeat(batch))
        want = want.cpu().numpy()
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= _step_of_four_bits(want)).all(), f"worst {(err / _step_of_four_bits(want)).max()}"


def test_positions_of_uneven_rows():
    lens = torch.tensor([7, 3, 9], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    assert D.Layer.positions(6, lens, starts).tolist() == [5, 6, 5, 6, 7, 8]
    assert D.Layer.positions(6, lens, None).tolist() == [5, 6, 1, 2, 7, 8]
