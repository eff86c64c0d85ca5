"""Refusals of the 8-bit, norm and rotary entry points, through the C ABI and without a GPU: a
bad call returns its status before anything is launched.  And the oracle's own format, and
the frequencies as fractions of a turn."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from entropy_coded_weight_amd import fp8
from tests import fp8_abi as A
from tests import fp8_ref as R

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 4
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    return A._lib()


def test_oracle_rounds_as_the_framework_of_the_tests_does():
    x = torch.cat([torch.arange(-448 * 32, 448 * 32 + 1).float() / 32, torch.arange(-300, 301).float() * 2 ** -12])
    want = x.to(torch.float8_e4m3fn).float().numpy()
    got = R.rounded(np.concatenate([np.full((len(x), 1), 448.0), x.numpy()[:, None].astype(np.float64)], 1))[:, 1]
    assert np.array_equal(got, want)
    assert R.LEVELS[-1] == 448 and R.LEVELS[1] == 2.0 ** -9


@pytest.mark.parametrize("top,byte", [(448.0, 127), (449.0, 128), (0.0, 127), (1.0, 119), (1.75, 119), (1.7500001, 120),
                                      (2.0 ** -126, 10), (3.4e38, 246), (float("inf"), 255), (float("nan"), 255)])
def test_oracle_scales(top, byte):
    assert R.quantise(np.array([[top, 0.0]]))[1][0, 0] == byte


@pytest.mark.parametrize("change,status", [
    ({"rows": 0}, OK), ({"cols": 0}, INVALID), ({"codes": 0}, INVALID), ({"codes": P + 8}, INVALID),
    ({"scales": P + 4}, INVALID), ({"x": 0}, INVALID), ({"x": P + 1}, INVALID), ({"dtype": ecw.DT_I8}, INVALID),
    ({"stride": -1}, INVALID), ({"gate": P + 1}, INVALID), ({"gate_stride": -1}, INVALID), ({"rows": 1 << 31}, INVALID),
    ({"cols": 1 << 31}, INVALID), ({"rows": 1 << 30, "cols": 1 << 30}, INVALID),
    ({"rows": 1 << 22, "cols": 1 << 13}, UNSUPPORTED)])
def test_quantize_and_dequantize(L, change, status):
    a = {"x": P, "dtype": ecw.DT_BF16, "stride": 64, "gate": 0, "gate_stride": 0, "rows": 2, "cols": 64, "codes": P,
         "scales": P, **change}
    assert L.fp8_quantize(None, a["x"], a["dtype"], a["stride"], a["gate"], a["gate_stride"], a["rows"], a["cols"],
                          a["codes"], a["scales"]) == status
    if not {"stride", "gate", "gate_stride"} & set(change):
        assert L.fp8_dequantize(None, a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["dtype"]) == status
    if status:
        assert L.ecw_last_error()


@pytest.mark.parametrize("change,status", [
    ({"batch": 0}, OK), ({"rows": 0}, OK), ({"cols": 0}, INVALID), ({"w": P + 8}, INVALID), ({"ws": 0}, INVALID),
    ({"x": 0}, INVALID), ({"xs": P + 1}, INVALID), ({"y": 0}, INVALID), ({"y": P + 8}, INVALID),
    ({"yd": ecw.DT_FP8_E4M3}, INVALID), ({"batch": 1 << 25}, INVALID), ({"rows": 1 << 31}, INVALID),
    ({"rows": 1 << 30, "batch": 1 << 20, "cols": 64}, UNSUPPORTED),
    ({"batch": 40, "rows": 64, "cols": 16384, "workspace": 0}, INVALID),
    ({"batch": 40, "rows": 64, "cols": 16384, "workspace": P + 8}, INVALID),
    ({"batch": 40, "rows": 64, "cols": 16384, "bytes": 40 * 64 * 4}, TOO_SMALL)])
def test_gemm(L, change, status):
    a = {"w": P, "ws": P, "rows": 16, "cols": 64, "x": P, "xs": P, "batch": 2, "y": P, "yd": ecw.DT_F32, "workspace": P,
         "bytes": 1 << 40, **change}
    assert L.fp8_gemm(None, a["w"], a["ws"], a["rows"], a["cols"], a["x"], a["xs"], a["batch"], a["y"], a["yd"],
                      a["workspace"], a["bytes"]) == status
    if status:
        assert L.ecw_last_error()


def test_gemm_workspace(L):
    """Parts of the columns for a few tiles only, a whole number of fp32 results each, and never
    more of them than CUs."""
    n = ctypes.c_size_t(7)
    for rows, cols, batch, yd in [(0, 64, 4, 1), (64, 64, 0, 1), (64, 4096, 1, 2), (4096, 4096, 4096, 2), (64, 128, 40, 3)]:
        assert L.fp8_gemm_workspace_size(rows, cols, batch, yd, n) == OK and n.value == 0
    for rows, cols, batch, yd in [(64, 16384, 40, 3), (63, 14336, 33, 2), (4096, 14336, 40, 3), (1000, 30000, 100, 1)]:
        assert L.fp8_gemm_workspace_size(rows, cols, batch, yd, n) == OK
        part = -(-rows * batch // 4) * 16
        assert n.value % part == 0 and 2 <= n.value // part <= 256
    for rows, cols, batch, yd in [(64, 0, 4, 1), (1 << 31, 64, 4, 1), (64, 64, 1 << 25, 1), (64, 64, 4, ecw.DT_I8)]:
        assert L.fp8_gemm_workspace_size(rows, cols, batch, yd, n) == INVALID
    assert L.fp8_gemm_workspace_size(64, 64, 4, 1, None) == INVALID


@pytest.mark.parametrize("change,status", [
    ({"rows": 0}, OK), ({"cols": 0}, INVALID), ({"cols": 32769}, UNSUPPORTED), ({"rows": 1 << 31}, INVALID),
    ({"x": 0}, INVALID), ({"x": P + 1}, INVALID), ({"y": 0}, INVALID), ({"y": P + 8}, INVALID), ({"y_scales": 0}, INVALID),
    ({"y_scales": P + 8}, INVALID), ({"weight": P + 1}, INVALID), ({"weight_dtype": ecw.DT_I8}, INVALID),
    ({"x_dtype": 0}, INVALID), ({"y_dtype": ecw.DT_I8}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": math.nan}, INVALID),
    ({"eps": math.inf}, INVALID), ({"residual": 0}, INVALID), ({"residual_out": 0}, INVALID), ({"residual": P + 2}, INVALID),
    ({"residual_out": P + 2}, INVALID), ({"residual_dtype": ecw.DT_F16}, UNSUPPORTED), ({"x_stride": -1}, INVALID),
    ({"residual_stride": -1}, INVALID), ({"residual_out_stride": 63}, INVALID), ({"residual_stride": 128}, INVALID),
    ({"residual_stride": 128, "rows": 0}, OK)])
def test_norm(L, change, status):
    a = {"x": P, "residual": P, "weight": P, "residual_out": P, "y": P, "y_scales": P, "x_stride": 64, "residual_stride": 64,
         "residual_out_stride": 64, "rows": 2, "cols": 64, "x_dtype": ecw.DT_BF16, "residual_dtype": ecw.DT_F32,
         "weight_dtype": ecw.DT_BF16, "y_dtype": ecw.DT_FP8_E4M3, "eps": 1e-6, **change}
    assert L.rms_norm(None, A.Norm(*a.values())) == status
    if status:
        assert L.ecw_last_error()
    assert L.rms_norm(None, None) == INVALID


@pytest.mark.parametrize("change,status", [
    ({"rows": 0}, OK), ({"q_heads": 0, "k_heads": 0}, OK), ({"head_dim": 0}, INVALID), ({"head_dim": 5000}, INVALID),
    ({"rotary_dim": 0}, INVALID), ({"rotary_dim": 7}, INVALID), ({"rotary_dim": 66}, INVALID), ({"axes": 0}, INVALID),
    ({"axes": 256}, INVALID), ({"rows": 1 << 30}, INVALID), ({"q_heads": 1 << 17}, INVALID), ({"dtype": ecw.DT_I8}, INVALID),
    ({"scale": math.inf}, INVALID), ({"freqs": 0}, INVALID), ({"freqs": P + 4}, INVALID), ({"axis_of": 0}, INVALID),
    ({"positions": 0}, INVALID), ({"positions": P + 2}, INVALID), ({"positions": P + 4, "wide_positions": 1}, INVALID),
    ({"q": 0}, INVALID), ({"q_out": P + 1}, INVALID), ({"k": P + 1}, INVALID), ({"k_out": 0}, INVALID),
    ({"q_row": -1}, INVALID), ({"axis_stride": -1}, INVALID), ({"q_out": P, "q_out_row": 128}, INVALID),
    ({"rows": 1 << 29, "q_heads": 4096}, UNSUPPORTED)])
def test_rotary(L, change, status):
    a = {"q": P, "k": P, "q_out": 2 * P, "k_out": 2 * P, "positions": P, "freqs": P, "axis_of": P, "q_row": 64, "q_head": 64,
         "k_row": 64, "k_head": 64, "q_out_row": 64, "q_out_head": 64, "k_out_row": 64, "k_out_head": 64, "axis_stride": 2,
         "rows": 2, "q_heads": 1, "k_heads": 1, "head_dim": 64, "rotary_dim": 64, "axes": 1, "dtype": ecw.DT_BF16,
         "neighbours": 0, "wide_positions": 0, "scale": 1.0, **change}
    assert L.rotary_apply(None, A.Rotary(*a.values())) == status
    if status:
        assert L.ecw_last_error()
    assert L.rotary_apply(None, None) == INVALID


@pytest.mark.parametrize("f", [1.0, 10000.0 ** -0.5, 1e-7, 6.25, -0.3, 0.0, 500000.0 ** (-62 / 64), 1e5])
def test_frequencies_as_fractions_of_a_turn(f):
    two_pi = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)
    want = Fraction(f) / two_pi
    want -= math.floor(want)
    got = Fraction(fp8._turn(f), 1 << 64)
    off = abs(got - want)
    assert min(off, 1 - off) <= Fraction(1, 1 << 65) + Fraction(1, 10 ** 35)


@pytest.mark.parametrize("kwargs", [
    {"head_dim": 0}, {"head_dim": 63}, {"head_dim": 64, "rotary_dim": 65}, {"head_dim": 64, "rotary_dim": 66},
    {"head_dim": 64, "base": 0.0}, {"head_dim": 64, "sections": [16, 8]}, {"head_dim": 64, "sections": [40, -8]},
    {"head_dim": 64, "axes": [0] * 31}, {"head_dim": 64, "axes": [-1] + [0] * 31}, {"head_dim": 64, "axes": [300] + [0] * 31},
    {"head_dim": 64, "sections": [32], "axes": [0] * 32}, {"head_dim": 64, "inv_freq": [1.0]},
    {"head_dim": 4, "inv_freq": [1.0, math.nan]}, {"head_dim": 4, "inv_freq": [1.0, math.inf]}])
def test_rotary_refuses_bad_shapes(kwargs):
    with pytest.raises(ValueError):
        ecw.Rotary(device="cpu", **kwargs)


def test_calls_refuse_tensors_off_the_gpu():
    x = torch.zeros(2, 64)
    for call in (lambda: ecw.fp8_quantize(x), lambda: ecw.rms_norm(x), lambda: ecw.rms_norm(x, out_dtype=torch.float8_e4m3fn),
                 lambda: ecw.rms_norm([1.0]), lambda: ecw.FP8Tensor(x, x, 2, 64), lambda: ecw.Rotary(64, device="cpu")):
        with pytest.raises(TypeError):
            call()


def test_short_sums_are_for_16_bit_outputs(L):
    short, n = 0x100, ctypes.c_size_t(7)
    args = (None, P, P, 16, 64, P, P, 0, P)
    for dt, status in ((ecw.DT_F16, OK), (ecw.DT_BF16, OK), (ecw.DT_F32, INVALID), (ecw.DT_I8, INVALID), (0, INVALID)):
        assert L.fp8_gemm(*args, dt | short, P, 1 << 40) == status
        assert L.fp8_gemm_workspace_size(16, 64, 0, dt | short, n) == status and n.value == 0
    assert L.fp8_gemm(*args, ecw.DT_F16 | 0x200, P, 1 << 40) == INVALID
    for dt in (ecw.DT_F16, ecw.DT_F16 | short):  # few tiles, many columns: parts either way
        assert L.fp8_gemm_workspace_size(64, 16384, 40, dt, n) == OK and n.value > 0
