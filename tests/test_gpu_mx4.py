"""The 4-bit quantiser and product on the GPU against their float64 definition.

Codes and scales are compared bit for bit.  Tolerance of a product: the products are
exact, so what is left is the fp32 sums, one rounding (at most 2^-23 of the running
magnitude, whatever the instruction's inner rounding) for each addition on a term's way:
up to 128 inside an instruction, one per instruction of 32 columns, 32 joins of waves
and scales; then half a step of the output type."""
import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from tests import mx4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


F64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _say(*a):
    print("[gpu]", *a, flush=True)


def _matrix(rows, cols, dtype, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randn(rows, 1, generator=g) * spread)
    return x.to(dtype).cuda()


def _parts(t):
    """Unpacked codes and scales up to the last block that holds a column."""
    blocks = -(-t.cols // 32)
    return R.unpack(t.codes.cpu().numpy())[:, : blocks * 32], t.scales.cpu().numpy()[:, :blocks]


def _check_quantised(x):
    t = ecw.mx4_quantize(x)
    codes, scales = _parts(t)
    want_c, want_s = R.quantise(F64(x))
    assert np.array_equal(scales, want_s)
    fine = np.repeat(scales != 255, 32, 1)
    assert np.array_equal(codes[fine], want_c[fine])
    pad = R.unpack(t.codes.cpu().numpy())[:, codes.shape[1]:]
    assert not pad.any(), "padding must hold zeros"
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 128), (7, 129), (33, 1000), (2, 4096),
                                       (300, 264)])
def test_quantize_bit_exact(rows, cols, dtype):
    _say("quantize", rows, cols, dtype)
    _check_quantised(_matrix(rows, cols, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_ties_limits_and_special_blocks(dtype):
    _say("quantize special", dtype)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 0.2490234375, 0.251953125, 4.0, 0.0])
    block = torch.cat([ties, -ties, torch.tensor([4.0, 0.5, 1.0, 3.0])])
    rows = [block * s for s in (1.0, 2.0 ** -9, 2.0 ** 5)]
    rows.append(torch.zeros(32))
    rows.append(-torch.zeros(32))
    for special in (float("inf"), -float("inf"), float("nan")):
        r = torch.ones(32)
        r[17] = special
        rows.append(r)
    if dtype != torch.float16:  # the ends of the scales' range, and below the smallest
        rows += [block * 2.0 ** 124, block * 2.0 ** -123, block * 2.0 ** -125, block * 2.0 ** -126,
                 torch.full((32,), torch.finfo(dtype).max), torch.full((32,), 2.0 ** -127)]
    else:
        rows += [torch.full((32,), 65504.0), torch.full((32,), 2.0 ** -24), block * 2.0 ** -20]
    x = torch.stack(rows).to(dtype).cuda()
    t = _check_quantised(x)
    for out in DTYPES:
        got, want = t.dequantize(out), R.rounded(F64(x))
        want = torch.from_numpy(want).to(out)
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0)), out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,offset,stride", [(100, 0, 104), (100, 3, 117), (64, 1, 64), (33, 0, 40)])
def test_quantize_rows_at_any_stride_and_alignment(cols, offset, stride, dtype):
    _say("quantize strided", cols, offset, stride, dtype)
    flat = _matrix(1, stride * 9 + offset + cols, dtype, seed=5, spread=0)[0]
    _check_quantised(flat.as_strided((9, cols), (stride, 1), offset))
    _check_quantised(flat.as_strided((4, cols), (0, 1), offset))  # a broadcast row


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (5, 128), (9, 1000), (4, 130)])
def test_dequantize(rows, cols, dtype):
    _say("dequantize", rows, cols, dtype)
    x = _matrix(rows, cols, torch.bfloat16, seed=2, spread=8.0)
    t = ecw.mx4_quantize(x)
    out = torch.full((rows * cols + 8,), 77.0, dtype=dtype, device="cuda")
    t.dequantize(dtype, out=out[: rows * cols].view(rows, cols))
    assert torch.equal(out[: rows * cols].view(rows, cols).cpu(), torch.from_numpy(R.rounded(F64(x))).to(dtype))
    assert bool((out[rows * cols:] == 77).all()), "written past the end"


def _check_product(w, x, y, xv=None):
    wv, xv = R.rounded(F64(w)), F64(x) if xv is None else xv
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    half = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[y.dtype]
    tiny = torch.finfo(y.dtype).smallest_normal * half
    tol = (128 + -(-w.shape[1] // 32) + 32) * 2.0 ** -23 * mag
    tol = tol + half * (np.abs(want) + tol) + tiny
    err = np.abs(F64(y) - want)
    assert y.shape == want.shape and (err <= tol).all(), f"worst {np.nanmax(err / tol)}"


PRODUCTS = [(1, 16, 32), (1, 1, 1), (1, 4096, 4096), (2, 40, 130), (3, 17, 100), (5, 1000, 333), (16, 64, 512),
            (17, 48, 129), (31, 257, 640), (33, 80, 96), (64, 128, 128), (100, 300, 1000), (129, 130, 257),
            (257, 513, 384), (300, 255, 2049)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("acts", ["bf16", "fp16", "mx4"])
@pytest.mark.parametrize("batch,rows,cols", PRODUCTS)
def test_gemm(batch, rows, cols, acts, out):
    _say("gemm", batch, rows, cols, acts, out)
    w = _matrix(rows, cols, torch.bfloat16, seed=1, spread=1.0) * 0.02
    x = _matrix(batch, cols, torch.float16 if acts == "fp16" else torch.bfloat16, seed=3, spread=1.0)
    t = ecw.mx4_quantize(w)
    if acts == "mx4":
        _check_product(w, x, t.gemm(ecw.mx4_quantize(x), out_dtype=out), R.rounded(F64(x)))
    else:
        _check_product(w, x, t.gemm(x, out_dtype=out))


@pytest.mark.parametrize("batch", [1, 7, 130])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gemm_scales_far_apart(batch, dtype):
    """Blocks of one row 2^40 apart, with x as uneven the other way: no block may vanish."""
    _say("gemm far scales", batch, dtype)
    w = _matrix(50, 512, torch.float32, seed=7, spread=0)
    w.view(50, 16, 32)[:, ::3] *= 2.0 ** -40
    w.view(50, 16, 32)[10:20] *= 0.0
    x = _matrix(batch, 512, torch.float32, seed=8, spread=0)
    x.view(batch, 16, 32)[:, 1::3] *= 2.0 ** -13
    x.view(batch, 16, 32)[:, 2::3] = 0
    x.view(batch, 16, 32)[:, 1::3] *= 0 if batch == 7 else 1
    x = x.to(dtype)
    _check_product(w, x, ecw.mx4_quantize(w).gemm(x))


@pytest.mark.parametrize("batch", [2, 40, 140])
@pytest.mark.parametrize("acts", ["bf16", "fp16", "mx4"])
def test_gemm_special_values_stay_in_their_rows(batch, acts):
    _say("gemm special", batch, acts)
    w = _matrix(70, 200, torch.float32, seed=1, spread=0)
    w[5, 190] = float("nan")
    w[66, 0] = float("inf")
    x = _matrix(batch, 200, torch.float16 if acts == "fp16" else torch.bfloat16, seed=2, spread=0)
    x[1, 3] = float("inf")
    t = ecw.mx4_quantize(w)
    y = t.gemm(ecw.mx4_quantize(x) if acts == "mx4" else x).cpu()
    bad_rows, keep_x = torch.zeros(70, dtype=torch.bool), torch.ones(batch, dtype=torch.bool)
    bad_rows[[5, 66]] = True
    keep_x[1] = False
    assert bool(torch.isnan(y[keep_x][:, bad_rows]).all())
    assert bool((~torch.isfinite(y[1])).all())
    assert bool(torch.isfinite(y[keep_x][:, ~bad_rows]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,cols,offset,stride", [(3, 100, 0, 104), (5, 96, 1, 101), (20, 300, 4, 306), (4, 64, 0, 0),
                                                      (150, 200, 0, 208), (150, 130, 3, 139)])
def test_gemm_rows_at_any_stride_and_alignment(batch, cols, offset, stride, dtype):
    _say("gemm strided", batch, cols, offset, stride, dtype)
    flat = torch.full((stride * batch + offset + cols + 16,), float("nan"), dtype=dtype, device="cuda")
    x = flat.as_strided((batch, cols), (stride, 1), offset)
    if stride:
        x.copy_(_matrix(batch, cols, dtype, seed=4, spread=0))  # NaN between and behind the rows
    else:
        flat[:cols + offset] = 0.5
    w = _matrix(66, cols, torch.bfloat16, seed=1, spread=0)
    _check_product(w, x, ecw.mx4_quantize(w).gemm(x))


def test_empty_sizes_launch_nothing():
    w = ecw.mx4_quantize(_matrix(8, 64, torch.bfloat16))
    assert w.gemm(torch.zeros(0, 64, dtype=torch.float16, device="cuda")).shape == (0, 8)
    none = ecw.mx4_quantize(torch.zeros(0, 64, device="cuda"))
    assert none.gemm(torch.zeros(3, 64, dtype=torch.float16, device="cuda")).shape == (3, 0)
    assert none.dequantize().shape == (0, 64)
    assert w.gemm(none).shape == (0, 8)


def test_vector_and_given_output():
    w = _matrix(40, 96, torch.bfloat16, seed=1)
    x = _matrix(1, 96, torch.bfloat16, seed=2)
    t = ecw.mx4_quantize(w)
    y = torch.full((1, 40), 9.0, device="cuda")
    assert t.gemm(x[0], y=y) is y
    _check_product(w, x, y)
    again = ecw.mx4_quantize(_matrix(40, 96, torch.bfloat16, seed=9), out=t)
    assert again is t
    _check_product(_matrix(40, 96, torch.bfloat16, seed=9), x, t.gemm(x))


def test_large_weight_offsets_pass_32_bits():
    """2^33 elements: byte offsets of the last rows' codes exceed 32 bits."""
    rows, cols = (1 << 17) + 40, 1 << 16
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    w = _matrix(40, cols, torch.bfloat16, seed=1, spread=0)
    small = ecw.mx4_quantize(w)
    codes[-40:], scales[-40:] = small.codes, small.scales
    t = ecw.MX4Tensor(codes, scales, rows, cols)
    for batch in (2, 130):
        x = _matrix(batch, cols, torch.bfloat16, seed=2, spread=0)
        for a in (x, ecw.mx4_quantize(x)):
            _say("gemm large", batch, type(a).__name__)
            y = t.gemm(a)
            _check_product(w, x, y[:, -40:], None if a is x else R.rounded(F64(x)))
            assert not y[:, :-40].any()


def test_another_stream():
    s = torch.cuda.Stream()
    w, x = _matrix(256, 512, torch.bfloat16, seed=1), _matrix(5, 512, torch.bfloat16, seed=2)
    torch.cuda.synchronize()
    t = ecw.mx4_quantize(w, stream=s)
    y = t.gemm(x, stream=s)
    z = t.gemm(ecw.mx4_quantize(x, stream=s), stream=s)
    d = t.dequantize(torch.bfloat16, stream=s)
    s.synchronize()
    _check_product(w, x, y)
    _check_product(w, x, z, R.rounded(F64(x)))
    assert np.array_equal(F64(d), R.rounded(F64(w)))


def test_graph_replays():
    w, x = _matrix(256, 512, torch.bfloat16, seed=1), _matrix(5, 512, torch.bfloat16, seed=2)
    t = ecw.mx4_quantize(w)
    t.gemm(ecw.mx4_quantize(x))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, z = t.gemm(x), t.gemm(ecw.mx4_quantize(x))
    for seed in range(4):
        x.copy_(_matrix(5, 512, torch.bfloat16, seed=10 + seed))
        want = t.gemm(x).clone(), t.gemm(ecw.mx4_quantize(x)).clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_same_result_every_time():
    w, x = _matrix(4096, 4096, torch.bfloat16, seed=1), _matrix(9, 4096, torch.float16, seed=2)
    t = ecw.mx4_quantize(w)
    first = t.gemm(x)
    for _ in range(5):
        assert torch.equal(t.gemm(x), first)


def test_refusals():
    w = ecw.mx4_quantize(_matrix(16, 64, torch.bfloat16))
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    for bad, error in ((x.float(), TypeError), (x[:, :32], ValueError), (x.cpu(), TypeError), (x[None], ValueError),
                       (torch.zeros(64, 2, dtype=torch.bfloat16, device="cuda").t(), TypeError)):
        with pytest.raises(error):
            w.gemm(bad)
    with pytest.raises(ValueError):
        w.gemm(ecw.mx4_quantize(x[:, :32].contiguous()))
    with pytest.raises(TypeError):
        w.gemm(x, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        w.gemm(x, y=torch.empty(2, 17, device="cuda"))
    with pytest.raises(TypeError):
        ecw.mx4_quantize(x.double())
    with pytest.raises(ValueError):
        ecw.mx4_quantize(torch.zeros(4, 0, device="cuda"))
    with pytest.raises(ValueError):
        ecw.mx4_quantize(x, out=w)
    with pytest.raises(ValueError):
        ecw.MX4Tensor(w.codes, w.scales, 16, 200)


@pytest.mark.parametrize("acts", ["bf16", "fp16", "mx4"])
@pytest.mark.parametrize("batch,rows,cols", [(5, 4100, 160), (12, 8200, 96), (40, 4112, 200), (70, 16400, 128),
                                             (200, 8200, 264), (260, 16500, 136), (600, 12400, 72), (1100, 8300, 40)])
def test_gemm_every_tile_size(batch, rows, cols, acts):
    """Sizes on both sides of each rule that picks a tile."""
    _say("gemm tiles", batch, rows, cols, acts)
    w = _matrix(rows, cols, torch.bfloat16, seed=1, spread=1.0)
    x = _matrix(batch, cols, torch.float16 if acts == "fp16" else torch.bfloat16, seed=3, spread=0)
    t = ecw.mx4_quantize(w)
    if acts == "mx4":
        _check_product(w, x, t.gemm(ecw.mx4_quantize(x)), R.rounded(F64(x)))
    else:
        _check_product(w, x, t.gemm(x))


def test_gemm_rows_far_apart():
    """Rows of x more than 2^31 bytes from the first."""
    _say("gemm far rows")
    flat = torch.zeros((1 << 30) * 2 + 512, dtype=torch.bfloat16, device="cuda")
    for batch in (3, 40):
        x = flat.as_strided((batch, 96), ((1 << 31) // batch // 8 * 8, 1))
        x.copy_(_matrix(batch, 96, torch.bfloat16, seed=3, spread=0))
        w = _matrix(50, 96, torch.bfloat16, seed=1, spread=0)
        _check_product(w, x, ecw.mx4_quantize(w).gemm(x))


def _loose(batch, cols, stride, dtype):
    """Rows that start at an odd element, with NaN before, between and behind them."""
    flat = torch.full((stride * batch + cols + 16,), float("nan"), dtype=dtype, device="cuda")
    x = flat.as_strided((batch, cols), (stride, 1), 1)
    return x.copy_(_matrix(batch, cols, dtype, seed=5, spread=0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [8, 9, 15, 127, 129, 250, 260, 391, 520, 645, 1151])
def test_gemm_rows_at_odd_elements(cols, dtype):
    """Last spans of every kind, and fewer spans than are asked for ahead."""
    for batch, rows in ((1, 40), (9, 70), (24, 70), (60, 70)):
        _say("gemm odd rows", batch, rows, cols, dtype)
        w, x = _matrix(rows, cols, torch.bfloat16, seed=1, spread=1.0), _loose(batch, cols, cols + 2, dtype)
        _check_product(w, x, ecw.mx4_quantize(w).gemm(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,rows,cols", [(40, 16400, 131), (70, 8200, 650), (70, 16400, 397), (200, 8200, 265),
                                             (200, 8200, 777), (260, 16500, 139), (260, 16500, 1030)])
def test_gemm_rows_at_odd_elements_every_tile_size(batch, rows, cols, dtype):
    _say("gemm odd rows, tiles", batch, rows, cols, dtype)
    w, x = _matrix(rows, cols, torch.bfloat16, seed=1, spread=1.0), _loose(batch, cols, cols, dtype)
    _check_product(w, x, ecw.mx4_quantize(w).gemm(x))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [1, 4, 7])
def test_gemm_narrow_rows(cols, dtype, out):
    _say("gemm narrow", cols, dtype, out)
    w, x = _matrix(300, cols, torch.bfloat16, seed=1, spread=1.0), _loose(33, cols, cols + 1, dtype)
    w[7, 0] = float("nan")
    y = ecw.mx4_quantize(w).gemm(x, out_dtype=out)
    assert y[:, 7].isnan().all()
    w, y = torch.cat([w[:7], w[8:]]), torch.cat([y[:, :7], y[:, 8:]], 1)
    _check_product(w, x, y)


@pytest.mark.parametrize("batch", [2, 12, 40, 140])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gemm_infinite_x_next_to_scales_far_apart(batch, dtype):
    """An infinity in x gives the definition's infinity or NaN in every output, whatever the
    neighbouring rows of w hold: close scales, far ones, a NaN block."""
    _say("gemm inf, far scales", batch, dtype)
    w = _matrix(70, 512, torch.float32, seed=7, spread=0)
    w[3, 64:96] *= 2.0 ** -40    # rows 0..15 next to a row of far scales
    w[20, 100] = float("nan")    # rows 16..31 next to a NaN block
    w.view(70, 16, 32)[40, ::2] *= 2.0 ** -30
    w[50:52] = 0                 # zeros times an infinity
    x = _matrix(batch, 512, dtype, seed=8, spread=0)
    x[0, 70], x[1, 5], x[1, 300] = float("inf"), -float("inf"), -float("inf")
    y = F64(ecw.mx4_quantize(w).gemm(x))
    with np.errstate(invalid="ignore"):
        want = F64(x) @ R.rounded(F64(w)).T
    assert np.array_equal(np.isnan(y), np.isnan(want)), "NaN elsewhere"
    inf = np.isinf(want)
    assert inf.any() and np.array_equal(y[inf], want[inf])
    keep = ~np.isin(np.arange(70), [20])
    _check_product(w[keep], x[2:], torch.from_numpy(y[2:][:, keep]).float())


@pytest.mark.parametrize("batch", [2, 40])
def test_gemm_every_nan_is_nan_next_to_scales_far_apart(batch):
    _say("gemm NaN payloads", batch)
    w = _matrix(33, 256, torch.float32, seed=7, spread=0)
    w[3, 64:96] *= 2.0 ** -40
    x = _matrix(batch, 256, torch.float16, seed=8, spread=0)
    for payload in (0x7c01, 0x7e00, 0x7fff, -0x3ff):  # signalling, quiet, all ones, negative
        x[1, 70].view(torch.int16).fill_(payload)
        y = ecw.mx4_quantize(w).gemm(x)
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[0]).all())


@pytest.mark.parametrize("acts", ["bf16", "fp16", "mx4"])
@pytest.mark.parametrize("batch,rows", [(4, 8300), (5, 8128), (5, 8130), (16, 8300), (17, 8300)])
def test_gemm_few_rows_by_a_long_k(batch, rows, acts):
    """Both sides of the rule between blocks of 16 rows and tiles, for long rows of w."""
    _say("gemm few, long", batch, rows, acts)
    w = _matrix(rows, 6400, torch.bfloat16, seed=1, spread=0)
    x = _matrix(batch, 6400, torch.float16 if acts == "fp16" else torch.bfloat16, seed=3, spread=0)
    t = ecw.mx4_quantize(w)
    if acts == "mx4":
        _check_product(w, x, t.gemm(ecw.mx4_quantize(x)), R.rounded(F64(x)))
    else:
        _check_product(w, x, t.gemm(x))
