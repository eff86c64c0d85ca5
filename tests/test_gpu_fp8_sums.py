"""Sums of the 8-bit product: fp32 for every output type and number of rows, and the short
ones that a caller may ask for, within their bound."""
import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from tests import fp8_ref as R
from tests.test_gpu_fp8 import DTYPES, SHAPES, _f64, _randn, _whole

pytestmark = pytest.mark.gpu
HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(autouse=True)
def _named(request):
    print(f"[gpu] {request.node.name}", flush=True)


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("batch,rows,cols", [(1, 48, 1024), (16, 64, 8192), (17, 80, 256), (40, 200, 4096), (70, 130, 640),
                                             (300, 520, 384), (1003, 700, 256), (2100, 1100, 128)])
def test_products_that_cancel(batch, rows, cols, out):
    """448^2 - 448^2 + 2^2 in every 16 columns is 4 each time; all are whole numbers under 2^24."""
    x, w = torch.zeros(batch, cols), torch.zeros(rows, cols)
    x[:, 0::16], x[:, 1::16], x[:, 2::16] = 448, 448, 2
    w[:, 0::16], w[:, 1::16], w[:, 2::16] = 448, -448, 2
    y = ecw.fp8_quantize(w.cuda()).gemm(ecw.fp8_quantize(x.cuda()), out_dtype=out)
    assert torch.equal(y.cpu(), torch.full((batch, rows), cols / 4).to(out))


def _real(batch, rows, cols, large):
    x, w = _randn(batch, cols, seed=4), _randn(rows, cols, seed=5)
    if large:
        x[:, ::50] *= 100
        w *= torch.exp2(3 * _randn(rows, 1, seed=6))
    xv, wv = R.rounded(x.double().numpy()), R.rounded(w.double().numpy())
    return ecw.fp8_quantize(x.cuda()), ecw.fp8_quantize(w.cuda()), xv @ wv.T, np.abs(xv) @ np.abs(wv).T


REAL = [(1, 1024, 4096), (6, 333, 14336), (16, 64, 8192), (40, 256, 5000), (130, 200, 2000), (513, 700, 1500)]


@pytest.mark.parametrize("batch,rows,cols", REAL)
@pytest.mark.parametrize("out", DTYPES)
def test_sums_are_fp32(batch, rows, cols, out):
    """`cols` exact products added in fp32, in any order and truncated or rounded: each addition is
    off by at most 2^-23 of the sums' magnitudes.  Then half a step of the output, of the sum.  A
    16-bit output is the fp32 one, whose sums are taken in the same order, rounded."""
    xt, wt, want, size = _real(batch, rows, cols, True)
    got, near = _f64(wt.gemm(xt, out_dtype=out)), cols * 2.0 ** -23 * size
    past = np.isinf(got)  # past the output's range (fp16: 65504): infinite there, of its own sign
    assert (np.abs(want) + near >= torch.finfo(out).max)[past].all() and (np.sign(got) == np.sign(want))[past].all()
    tol = near + torch.finfo(out).eps / 2 * (np.abs(want) + near) + torch.finfo(out).smallest_normal * torch.finfo(out).eps
    assert (np.abs(got - want) <= tol)[~past].all()
    assert np.array_equal(got, _f64(wt.gemm(xt).to(out)))


@pytest.mark.parametrize("batch,rows,cols", REAL)
@pytest.mark.parametrize("out", HALVES)
def test_short_sums(batch, rows, cols, out):
    """Each of 16 products may lose 2^-12 of the largest one's power of two: under 2^-8 of the sum of
    their magnitudes.  Of unit normal numbers the largest of 16 products is 3.5 in root mean square,
    so losses of either sign come to 3.5 * 2^-12 < 2^-10 of the result in 2-norm."""
    for large in (True, False):
        xt, wt, want, size = _real(batch, rows, cols, large)
        got, near = _f64(wt.gemm(xt, out_dtype=out, short_sums=True)), (2.0 ** -8 + cols * 2.0 ** -23) * size
        past = np.isinf(got)
        assert (np.abs(want) + near >= torch.finfo(out).max)[past].all() and (np.sign(got) == np.sign(want))[past].all()
        tol = near + torch.finfo(out).eps / 2 * (np.abs(want) + near)
        assert (np.abs(got - want) <= tol)[~past].all()
    assert np.linalg.norm(got - want) <= (2.0 ** -10 + torch.finfo(out).eps / 2) * np.linalg.norm(want)


@pytest.mark.parametrize("batch,rows,cols", SHAPES + [(2048, 9000, 256), (17, 20000, 257), (40, 100, 25000), (33, 63, 20000),
                                                      (130, 130, 16385), (1043, 14511, 1800), (538, 13235, 2300), (1000, 9000, 4000)])
def test_short_sums_of_whole_numbers_are_exact(batch, rows, cols):
    """Products of at most 3 * 3 * 4 need no more than six of the twelve bits, sums stay under 2^24:
    nothing is lost, in tiles of every kind, parts of the columns and rounds that are cut."""
    most = 3 if cols < 10000 else 1
    x, w = _whole(batch, cols, most, 1, 1).cuda(), _whole(rows, cols, most, 2, 1).cuda()
    want = x @ w.t()  # fp32 sums of the same whole numbers, exact too
    assert want.abs().max() < 2 ** 24
    xt, wt = ecw.fp8_quantize(x), ecw.fp8_quantize(w)
    for out in HALVES:
        assert torch.equal(wt.gemm(xt, out_dtype=out, short_sums=True), want.to(out))


def test_short_sums_are_refused_for_fp32():
    t = ecw.fp8_quantize(torch.ones(4, 256, device="cuda"))
    for y in (None, torch.zeros(4, 4, device="cuda")):
        with pytest.raises(ValueError):
            t.gemm(t, y, short_sums=True)
    assert (t.gemm(t, torch.zeros(4, 4, dtype=torch.float16, device="cuda"), short_sums=True) == 256).all()


# Both instructions, and 16-bit outputs of both.
SUMS = [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, False), (torch.float16, True)]
BATCHES = [1, 16, 17, 20, 70, 300]


@pytest.mark.parametrize("out,short", SUMS)
@pytest.mark.parametrize("batch", BATCHES)
def test_nan_blocks(batch, out, short):
    """A NaN block of w is NaN in its row's outputs, one of x in its own row; no others."""
    x, w = _whole(batch, 300, 3, 1), _whole(40, 300, 3, 2)
    x[batch - 1, 290], w[7, 5], w[39, 130] = float("inf"), float("nan"), float("-inf")
    y = ecw.fp8_quantize(w.cuda()).gemm(ecw.fp8_quantize(x.cuda()), out_dtype=out, short_sums=short).cpu()
    bad = torch.zeros(batch, 40, dtype=torch.bool)
    bad[batch - 1] = True
    bad[:, [7, 39]] = True
    assert torch.equal(torch.isnan(y), bad)
    x[batch - 1, 256:], w[7, :128], w[39, 128:256] = 0, 0, 0
    assert torch.equal(y[~bad], (x.double() @ w.double().t()).to(out)[~bad])


@pytest.mark.parametrize("out,short", SUMS)
@pytest.mark.parametrize("batch", BATCHES)
def test_nan_scales_over_numbers(batch, out, short):
    """The scale byte alone makes a block NaN, whatever its codes, zeros among them."""
    xv = _whole(batch, 300, 3, 1)
    xv[0, 256:] = 0
    x, w = ecw.fp8_quantize(xv.cuda()), ecw.fp8_quantize(_whole(40, 300, 3, 2).cuda())
    x.scales[0, 2] = 255
    w.scales[11, 0] = 255
    bad = torch.zeros(batch, 40, dtype=torch.bool)
    bad[0], bad[:, 11] = True, True
    assert torch.equal(torch.isnan(w.gemm(x, out_dtype=out, short_sums=short)).cpu(), bad)


@pytest.mark.parametrize("out,short", SUMS)
@pytest.mark.parametrize("batch", BATCHES)
def test_nan_codes(batch, out, short):
    """A code that is NaN beside numbers, with a scale of its block's: of either sign."""
    x, w = ecw.fp8_quantize(_whole(batch, 300, 3, 1).cuda()), ecw.fp8_quantize(_whole(40, 300, 3, 2).cuda())
    x.codes[batch - 1, 130], w.codes[3, 17], w.codes[38, 299] = 0x7f, 0xff, 0x7f
    bad = torch.zeros(batch, 40, dtype=torch.bool)
    bad[batch - 1], bad[:, [3, 38]] = True, True
    assert torch.equal(torch.isnan(w.gemm(x, out_dtype=out, short_sums=short)).cpu(), bad)


@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("batch", BATCHES)
def test_ends_of_the_range(batch, short):
    """Scales at both ends of their range: sums that pass fp32 are infinite, of their own sign,
    products under it vanish, and what lies between is exact."""
    def product(a, b):
        return ecw.fp8_quantize(torch.full((32, 256), b, device="cuda")).gemm(
            ecw.fp8_quantize(torch.full((batch, 256), a, device="cuda")), out_dtype=torch.bfloat16, short_sums=short).cpu()
    v = R.rounded(np.full((1, 256), np.float64(np.float32(3e38))))[0, 0]
    assert torch.equal(product(3e38, 2.0 ** -100), torch.full((batch, 32), v * 2.0 ** -100 * 256, dtype=torch.float64).bfloat16())
    assert torch.equal(product(2.0 ** -117, 2.0 ** 100), torch.full((batch, 32), 2.0 ** -9, dtype=torch.bfloat16))
    assert (product(3e38, 3e38) == float("inf")).all() and (product(-3e38, 3e38) == float("-inf")).all()
    assert (product(2.0 ** -100, 2.0 ** -100) == 0).all()


@pytest.mark.parametrize("out,short", SUMS)
@pytest.mark.parametrize("batch", [3, 40, 300])
def test_two_streams_and_two_graphs_at_once(batch, out, short):
    """Calls that overlap share nothing: the same weights on two streams, and two graphs of them
    replayed in turn."""
    w = ecw.fp8_quantize(_whole(100, 20000, 1, 1).cuda())
    xs = [ecw.fp8_quantize(_whole(batch, 20000, 1, 2 + i).cuda()) for i in range(2)]
    want = [w.gemm(x).to(out) for x in xs]  # whole numbers, exact in every order
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[w.gemm(xs[i], out_dtype=out, short_sums=short, stream=streams[i]) for i in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for turn in got for i, y in enumerate(turn))
    graphs, held = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            held.append(w.gemm(xs[i], out_dtype=out, short_sums=short))
    for _ in range(3):
        for y in held:
            y.zero_()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                streams[i].wait_stream(torch.cuda.default_stream())
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(held[i], want[i]) for i in range(2))
