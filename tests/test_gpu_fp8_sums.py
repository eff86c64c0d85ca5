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
