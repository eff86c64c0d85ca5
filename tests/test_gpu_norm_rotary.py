"""The root-mean-square norm and the rotary positions against their definitions in float64."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from tests import fp8_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]
EIGHT = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(autouse=True)
def _named(request):
    print(f"[gpu] {request.node.name}", flush=True)


def _randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ norm
# In fp32: h rounded once (its square twice that), the sum of squares by up to 32 products a
# lane in order and 10 additions of a tree, mean, root and reciprocal, two multiplications: the
# factor is off by half of (2 + 42 + 2) roundings of 2^-24 and 2 more, the result by 4 more of
# its own: under 32 * 2^-24.
NEAR = 2.0 ** -19


def _check_norm(x, weight, residual, eps, dtype, **kwargs):
    got = ecw.rms_norm(x, weight, residual=residual, eps=eps, out_dtype=dtype, **kwargs)
    y, h = got if residual is not None else (got, None)
    want, wide = R.norm(_f64(x), None if weight is None else _f64(weight), None if residual is None else _f64(residual), eps)
    if dtype is EIGHT:
        v = _f64(y.dequantize(torch.float32))
        # h itself is rounded: where x and residual cancel, by 2^-24 of the sum's own size
        assert R.between(v, want, NEAR).all()
        assert (y.scales.cpu().numpy()[:, -(-x.shape[-1] // 128):] == 127).all()
    else:
        dtype = dtype or x.dtype
        assert y.dtype == dtype and y.shape == x.shape
        tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        err = np.abs(_f64(y) - want)
        assert (err <= (NEAR + torch.finfo(dtype).eps / 2) * np.abs(want) + tiny).all(), f"worst {err.max()}"
    if h is not None:
        assert h.dtype == residual.dtype
        assert torch.equal(h, (x.float() + residual.float()).to(residual.dtype))
    return y, h


COLS = [1, 2, 7, 8, 9, 15, 64, 100, 127, 128, 129, 135, 500, 512, 520, 1000, 2047, 2048, 2056, 4095, 4096, 4104, 8192, 8200,
        16384, 16385, 20001, 32768]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype,res", [(torch.bfloat16, None), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                       (torch.float32, torch.float32)])
def test_norm(cols, dtype, res):
    for rows in (1, 3, 37):
        x = _randn(rows, cols, seed=cols, dtype=dtype)
        w = 1 + 0.3 * _randn(cols, seed=2, dtype=torch.float32)
        r = None if res is None else (5 * _randn(rows, cols, seed=3)).to(res)
        _check_norm(x, w.to(dtype), r, 1e-6, EIGHT)
        _check_norm(x, w, r, 1e-5, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", DTYPES + [EIGHT])
def test_norm_types(dtype, out):
    for res in (None, dtype, torch.float32):
        for wt in (None, *DTYPES):
            x = _randn(5, 300, seed=1, dtype=dtype)
            w = None if wt is None else _randn(300, seed=2, dtype=wt)
            _check_norm(x, w, None if res is None else _randn(5, 300, seed=3, dtype=res), 1e-6, out)


@pytest.mark.parametrize("rows,cols", [(33000, 16), (33001, 128), (9000, 512), (2500, 1024), (2100, 4096), (700, 9000)])
def test_norm_of_many_rows(rows, cols):
    """More rows than the launch has blocks for at once."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    r = torch.randn(rows, cols, generator=g, device="cuda")
    _check_norm(x, None, r, 1e-6, EIGHT)
    _check_norm(x, None, None, 1e-6, None)


def test_norm_strides_offsets_and_in_place():
    big, res = _randn(20, 700, seed=1, dtype=torch.bfloat16), _randn(20, 900, seed=2, dtype=torch.float32)
    for x, r in ((big[:, 1:334], res[:, 3:336]), (big[::2, 3:], res[:10, 5:702]), (big[:1, :200].expand(6, 200), res[:6, 1:201]),
                 (big[2:8, 9:10], res[:6, :1].expand(6, 1)), (big[0:5, 8:520], res[1:2, 8:520].expand(5, 512)), (big[3, 7:400], res[1, :393])):
        for dtype in (EIGHT, None):
            if x.dim() == 1 and dtype is EIGHT:
                t, h = ecw.rms_norm(x, residual=r, out_dtype=EIGHT)
                assert t.shape == (1, 393) and h.shape == (393,)
                continue
            _check_norm(x, None, r, 1e-6, dtype)
    # the residual in place, inside a wider tensor whose other columns stay
    x, r = big[:, 8:520].clone(), res.clone()
    want = (x.float() + r[:, 3:515]).clone()
    y, h = ecw.rms_norm(x, residual=r[:, 3:515], residual_out=r[:, 3:515])
    assert torch.equal(r[:, 3:515], want) and h.data_ptr() == r[:, 3:].data_ptr()
    assert torch.equal(r[:, :3], res[:, :3]) and torch.equal(r[:, 515:], res[:, 515:])
    # the result over x, and the new residual over x
    z = x.clone()
    assert ecw.rms_norm(z, out=z) is not None and torch.equal(z, ecw.rms_norm(x))
    z, r = x.float(), res[:, 3:515].clone()
    y2, h2 = ecw.rms_norm(z, residual=r, residual_out=z)
    assert torch.equal(z, want) and torch.equal(r, res[:, 3:515])
    # given outputs
    t = ecw.rms_norm(x, out_dtype=EIGHT)
    given = ecw.FP8Tensor(torch.zeros_like(t.codes), torch.zeros_like(t.scales), *t.shape)
    assert ecw.rms_norm(x, out=given) is given and torch.equal(given.codes, t.codes) and torch.equal(given.scales, t.scales)


def test_norm_of_zeros_infinities_and_nan():
    """A row's NaN stays in its row; a row of zeros is zeros (with eps) or NaN (without)."""
    x = _randn(6, 200, seed=1)
    x[1], x[2, 5], x[3, 7], x[5] = 0, float("inf"), float("nan"), 1e-25
    y = ecw.rms_norm(x, eps=1e-6)
    assert torch.isfinite(y[[0, 1, 4, 5]]).all() and (y[1] == 0).all() and torch.isnan(y[3]).all()
    assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all()
    assert torch.allclose(y[5], torch.full_like(y[5], 1e-22), rtol=1e-5)
    assert torch.isnan(ecw.rms_norm(x, eps=0.0)[1]).all()
    t = ecw.rms_norm(x, eps=1e-6, out_dtype=EIGHT).dequantize(torch.float32)
    assert torch.isfinite(t[[0, 1, 4, 5]]).all() and torch.isnan(t[3]).all() and torch.isnan(t[2, :128]).all() and (t[2, 128:] == 0).all()


def test_norm_with_infinite_and_nan_weights():
    """A weight that is infinite makes its column infinite, with the sign of its number; NaN its column NaN."""
    x = _randn(3, 300, seed=1).abs() + 0.5
    w = torch.ones(300, device="cuda")
    w[7], w[8], w[200] = float("inf"), float("-inf"), float("nan")
    y = ecw.rms_norm(x, w)
    assert (y[:, 7] == float("inf")).all() and (y[:, 8] == float("-inf")).all() and torch.isnan(y[:, 200]).all()
    rest = torch.ones(300, dtype=torch.bool)
    rest[[7, 8, 200]] = False
    assert torch.equal(y[:, rest], ecw.rms_norm(x)[:, rest])
    t = ecw.rms_norm(x, w, out_dtype=EIGHT).dequantize(torch.float32)
    assert torch.isnan(t[:, :256]).all() and torch.isfinite(t[:, 256:]).all()


def test_norm_far_from_one():
    """Numbers and factors near the ends of what squares in fp32 hold."""
    x = _randn(4, 500, seed=1)
    for size, eps in ((1e18, 1e-6), (1e-17, 0.0), (1e-18, 1e-38), (1.0, 1e30)):
        _check_norm(x * size, None, None, eps, torch.float32)
        _check_norm(x * size, None, x * size, eps, EIGHT)


def test_norm_offsets_past_32_bits():
    rows, cols = 132000, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = _randn(3, cols, seed=1).bfloat16()
    y, h = ecw.rms_norm(x, residual=x)
    want, wide = ecw.rms_norm(x[-3:], residual=x[-3:])
    assert torch.equal(y[-3:], want) and torch.equal(h[-3:], wide)
    del y, h
    t, n = ecw.rms_norm(x, out_dtype=EIGHT), ecw.rms_norm(x[-3:], out_dtype=EIGHT)
    assert torch.equal(t.codes[-3:], n.codes) and torch.equal(t.scales[-3:], n.scales)


def test_norm_empty_and_refusals():
    x, w = torch.ones(4, 256, device="cuda"), torch.ones(256, device="cuda")
    assert ecw.rms_norm(x[:0], w).shape == (0, 256) and ecw.rms_norm(x[:0], out_dtype=EIGHT).shape == (0, 256)
    y, h = ecw.rms_norm(x[:0], residual=x[:0])
    assert y.shape == h.shape == (0, 256)
    t = ecw.fp8_quantize(x)
    for call, error in [
            (lambda: ecw.rms_norm(x.double()), TypeError), (lambda: ecw.rms_norm(x.t()), TypeError),
            (lambda: ecw.rms_norm(x[None]), ValueError), (lambda: ecw.rms_norm(x[:, :0]), ValueError),
            (lambda: ecw.rms_norm(x, w[:5]), ValueError), (lambda: ecw.rms_norm(x, w.cpu()), TypeError),
            (lambda: ecw.rms_norm(x, w.int()), TypeError), (lambda: ecw.rms_norm(x, w, eps=-1.0), ecw.EcwError),
            (lambda: ecw.rms_norm(x, residual=x[:2]), ValueError), (lambda: ecw.rms_norm(x, residual=x.half()), TypeError),
            (lambda: ecw.rms_norm(x, residual_out=x), ValueError),
            (lambda: ecw.rms_norm(x, residual=x, residual_out=x.half()), ValueError),
            (lambda: ecw.rms_norm(x, residual=x.clone(), residual_out=x[:1].expand(4, 256)), ValueError),
            (lambda: ecw.rms_norm(x[1:], residual=x[1:].clone(), residual_out=x[:3]), ValueError),
            (lambda: ecw.rms_norm(x, residual=x.clone(), out=x, residual_out=x), ValueError),
            (lambda: ecw.rms_norm(x, w, out=x[:3]), ValueError), (lambda: ecw.rms_norm(x[:3], out=x[1:]), ValueError),
            (lambda: ecw.rms_norm(x, out=x, out_dtype=EIGHT), TypeError), (lambda: ecw.rms_norm(x[:2], out=t), ValueError),
            (lambda: ecw.rms_norm(x, out_dtype=torch.int8), TypeError),
            (lambda: ecw.rms_norm(torch.ones(1, 40000, device="cuda")), ecw.EcwError)]:
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------ rotary
_TWO_PI = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)


def _angles(positions, inv_freq, axes):
    """cos and sin [rows, pairs] in float64, the angle reduced exactly."""
    p = positions.cpu().numpy().reshape(-1, positions.shape[-1])
    out = np.zeros((p.shape[1], len(inv_freq)))
    for j, f in enumerate(inv_freq):
        step = Fraction(float(f))
        for i, x in enumerate(p[axes[j]]):
            turn = int(x) * step / _TWO_PI
            out[i, j] = float(turn - math.floor(turn)) * 2 * math.pi
    return np.cos(out), np.sin(out)


def _check_rotary(rotary, q, k, positions, inv_freq, axes, got=None):
    """Sine and cosine are within 2^-23, the two products and their sum add 2^-24 of the terms
    each, times the scale; then half a step of the output's type."""
    cos, sin = _angles(positions, inv_freq, axes)
    got = rotary(q, k, positions) if got is None else got
    got = got if isinstance(got, tuple) else (got,)
    for x, y in zip((q, k), got):
        assert y.dtype == x.dtype and y.shape == x.shape
        want = R.rotate(_f64(x), cos * rotary.scale, sin * rotary.scale, rotary.rotary_dim, rotary.neighbours)
        size = R.rotate(np.abs(_f64(x)), np.ones_like(cos), -np.ones_like(sin), rotary.rotary_dim, rotary.neighbours)
        size = np.maximum(size, R.rotate(np.abs(_f64(x)), np.ones_like(cos), np.ones_like(sin), rotary.rotary_dim, rotary.neighbours))
        e = np.abs(_f64(y) - want)
        tol = abs(rotary.scale) * 2.0 ** -21.5 * size + torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -140
        if x.dtype == torch.float16:
            tol = tol + 2.0 ** -25
        tol[..., rotary.rotary_dim:] = 0
        assert (e <= tol).all(), f"worst {(e / np.maximum(tol, 1e-300)).max()}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("dim,part", [(2, 2), (6, 6), (6, 2), (64, 64), (80, 80), (80, 20), (96, 96), (128, 128), (128, 64),
                                      (128, 34), (192, 192), (256, 256), (31, 30), (100, 14)])
def test_rotary(dtype, neighbours, dim, part):
    rows = 5
    q, k = _randn(rows, 6, dim, seed=1, dtype=dtype), _randn(rows, 2, dim, seed=2, dtype=dtype)
    inv = [10000.0 ** (-2 * j / part) for j in range(part // 2)]
    positions = torch.tensor([0, 1, 77, 131071, 1048575], dtype=torch.int32, device="cuda")
    r = ecw.Rotary(dim, rotary_dim=part, neighbours=neighbours)
    _check_rotary(r, q, k, positions, inv, [0] * (part // 2))
    one = r(q, None, positions)
    assert isinstance(one, torch.Tensor) and torch.equal(one, r(q, k, positions)[0])


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotary_axes_and_positions(neighbours):
    """Axes by sections and by pair, far and negative positions, 64-bit ones, own frequencies
    and a scale."""
    dim, rows = 96, 7
    q, k = _randn(rows, 3, dim, seed=1), _randn(rows, 1, dim, seed=2)
    inv = [500000.0 ** (-2 * j / dim) for j in range(48)]
    at = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, rows), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    at[:, 0] = 0
    _check_rotary(ecw.Rotary(dim, base=500000.0, sections=[8, 20, 20], neighbours=neighbours), q, k, at, inv, [0] * 8 + [1] * 20 + [2] * 20)
    axes = [j % 3 for j in range(48)]
    own = [6.5 * 0.9 ** j for j in range(48)]
    _check_rotary(ecw.Rotary(dim, inv_freq=own, axes=axes, neighbours=neighbours, scale=0.7), q, k, at, own, axes)
    _check_rotary(ecw.Rotary(dim, inv_freq=torch.tensor(own), axes=axes, neighbours=neighbours), q, k, at, np.float32(own), axes)
    wide = torch.randint(-2 ** 62, 2 ** 62, (2, rows), generator=torch.Generator().manual_seed(2)).cuda()
    wide //= torch.tensor([2 ** 22], device="cuda")  # up to 2^40
    _check_rotary(ecw.Rotary(dim, inv_freq=own, axes=[j % 2 for j in range(48)], neighbours=neighbours), q, k, wide, own, [j % 2 for j in range(48)])
    assert torch.equal(ecw.Rotary(dim)(q, None, at[:1].long()), ecw.Rotary(dim)(q, None, at[0]))
    # sections with an empty axis
    _check_rotary(ecw.Rotary(dim, base=500000.0, sections=[0, 48, 0], neighbours=neighbours), q, k, at, inv, [1] * 48)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,q_heads,k_heads,dim", [(1, 32, 8, 128), (3000, 5, 3, 128), (700, 40, 8, 64), (5000, 33, 1, 64)])
def test_rotary_of_many_rows_is_that_of_each(dtype, rows, q_heads, k_heads, dim):
    """Any number of rows and heads gives the bits that a row and a head by itself does."""
    q, k = _randn(rows, q_heads, dim, seed=1, dtype=dtype), _randn(rows, k_heads, dim, seed=2, dtype=dtype)
    at = torch.randint(0, 100000, (rows,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    r = ecw.Rotary(dim)
    a, b = r(q, k, at)
    pick = torch.tensor(sorted({0, rows // 3, rows - 1}))
    _check_rotary(r, q[pick], k[pick], at[pick], [10000.0 ** (-2 * j / dim) for j in range(dim // 2)], [0] * (dim // 2), (a[pick], b[pick]))
    for h in (0, q_heads - 1):
        assert torch.equal(r(q[:, h:h + 1], None, at), a[:, h:h + 1])
    assert torch.equal(r(k[:, -1:], None, at), b[:, -1:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_rotary_strides_and_in_place(dtype):
    """q and k as parts of one projection's rows, odd offsets, and results written over them."""
    dim, rows = 64, 9
    qkv = _randn(rows, 1 + (4 + 2 + 2) * dim, seed=1, dtype=dtype)
    at = torch.arange(rows, dtype=torch.int64, device="cuda") * 1000
    for off in (0, 1):
        for part in (64, 20):
            r = ecw.Rotary(dim, rotary_dim=part)
            x = qkv.clone()
            q, k = x[:, off:off + 4 * dim].view(rows, 4, dim), x[:, off + 4 * dim:off + 6 * dim].view(rows, 2, dim)
            want = r(q.contiguous(), k.contiguous(), at)
            for g, w in zip(r(q, k, at), want):
                assert torch.equal(g, w) and g.is_contiguous()
            got = r(q, k, at, out=(q, k))
            assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
            assert torch.equal(x[:, off + 6 * dim:], qkv[:, off + 6 * dim:]) and torch.equal(x[:, :off], qkv[:, :off])
            y = torch.zeros(rows, 4, 2 * dim, dtype=dtype, device="cuda")
            r(qkv[:, off:off + 4 * dim].view(rows, 4, dim), None, at, out=y[:, :, dim:])
            assert torch.equal(y[:, :, dim:], want[0]) and (y[:, :, :dim] == 0).all()
    shared = qkv[:1, :dim].view(1, 1, dim).expand(rows, 3, dim)
    assert torch.equal(ecw.Rotary(dim)(shared, None, at), ecw.Rotary(dim)(shared.contiguous(), None, at))


def test_rotary_offsets_past_32_bits():
    rows, heads, dim = 270000, 128, 128
    q = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[-2:] = _randn(2, heads, dim, seed=1).bfloat16()
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    r = ecw.Rotary(dim)
    want = r(q[-2:].clone(), None, at[-2:])
    r(q, None, at, out=q)
    assert torch.equal(q[-2:], want)


def test_rotary_undone_by_negated_positions():
    q = _randn(20, 2, 128, seed=1)
    at = torch.randint(0, 1 << 30, (20,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    r = ecw.Rotary(128)
    assert (r(r(q, None, at), None, -at) - q).abs().max() <= 2.0 ** -20 * q.abs().max()


def test_rotary_empty_and_refusals():
    r = ecw.Rotary(64, sections=[10, 22])
    q, k = torch.ones(3, 2, 64, device="cuda"), torch.ones(3, 1, 64, device="cuda")
    at = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    assert r(q[:0], k[:0], at[:, :0])[0].shape == (0, 2, 64)
    assert r(q[:, :0], k, at)[0].shape == (3, 0, 64)
    for call, error in [
            (lambda: r(q[0], k, at), ValueError), (lambda: r(q[..., :32], k, at), ValueError), (lambda: r(q, k[:2], at), ValueError),
            (lambda: r(q, k.half(), at), ValueError), (lambda: r(q.double(), None, at), TypeError), (lambda: r(q, k, at[0]), ValueError),
            (lambda: r(q, k, at[:, :2]), ValueError), (lambda: r(q, k, at.float()), TypeError), (lambda: r(q, k, at.cpu()), TypeError),
            (lambda: r(q.cpu(), k, at), TypeError), (lambda: r(q, k, at, out=(q[:2], k)), ValueError),
            (lambda: r(q, k, at, out=(k.expand(3, 2, 64), k)), ValueError), (lambda: r(q, None, at, out=(q, k)), ValueError),
            (lambda: r(q[:, :1], q[:, 1:], at, out=(q[:, 1:], None)), ValueError),
            (lambda: r(q.transpose(0, 2).contiguous().transpose(0, 2), None, at), TypeError)]:
        with pytest.raises(error):
            call()


def test_streams_and_graphs():
    """Norm, product and rotation as they follow each other, on another stream and captured."""
    w = ecw.fp8_quantize(_randn(6 * 64, 256, seed=1))
    x, res = _randn(5, 256, seed=2, dtype=torch.bfloat16), _randn(5, 256, seed=3)
    at = torch.arange(5, dtype=torch.int32, device="cuda")
    r = ecw.Rotary(64)

    def run(stream=None):
        h, s = ecw.rms_norm(x, residual=res, out_dtype=EIGHT, stream=stream)
        y = w.gemm(h, out_dtype=torch.bfloat16, stream=stream).view(5, 6, 64)
        return (*r(y[:, :4], y[:, 4:], at, stream=stream), s)

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(3):
        x.copy_(_randn(5, 256, seed=10 + i, dtype=torch.bfloat16))
        at += 17
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
