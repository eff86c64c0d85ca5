"""Refusals of the 4-bit entry points, through the C ABI and without a GPU: a bad call
returns its status before anything is launched."""
import ctypes
import os
import sysconfig

import pytest
import torch

import entropy_coded_weight_amd as ecw
from tests import mx4_abi as mx4

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    return mx4._lib()


@pytest.mark.parametrize("change,status", [
    ({"rows": 0}, OK), ({"cols": 0}, INVALID), ({"codes": 0}, INVALID), ({"codes": P + 8}, INVALID),
    ({"scales": P + 4}, INVALID), ({"x": 0}, INVALID), ({"x": P + 1}, INVALID), ({"dtype": ecw.DT_I8}, INVALID),
    ({"stride": -1}, INVALID), ({"rows": 1 << 31}, INVALID), ({"cols": 1 << 31}, INVALID),
    ({"rows": 1 << 30, "cols": 1 << 30}, INVALID), ({"rows": 1 << 28, "cols": 1 << 14}, UNSUPPORTED)])
def test_quantize_and_dequantize(L, change, status):
    a = {"x": P, "dtype": ecw.DT_BF16, "stride": 64, "rows": 2, "cols": 64, "codes": P, "scales": P, **change}
    assert L.mx4_quantize(None, a["x"], a["dtype"], a["stride"], a["rows"], a["cols"], a["codes"], a["scales"]) == status
    if "stride" not in change:
        assert L.mx4_dequantize(None, a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["dtype"]) == status
    if status:
        assert L.ecw_last_error()


@pytest.mark.parametrize("change,status", [
    ({"batch": 0}, OK), ({"rows": 0}, OK), ({"cols": 0}, INVALID), ({"w": P + 8}, INVALID), ({"ws": 0}, INVALID),
    ({"x": 0}, INVALID), ({"x": P + 1}, INVALID), ({"y": 0}, INVALID), ({"y": P + 8}, INVALID),
    ({"xd": ecw.DT_F32}, INVALID), ({"yd": ecw.DT_I8}, INVALID), ({"stride": -8}, INVALID),
    ({"batch": 1 << 25}, INVALID), ({"rows": 1 << 31}, INVALID)])
def test_gemm(L, change, status):
    a = {"w": P, "ws": P, "rows": 16, "cols": 64, "x": P, "xd": ecw.DT_F16, "stride": 64, "batch": 2, "y": P,
         "yd": ecw.DT_F32, **change}
    assert L.mx4_gemm(None, a["w"], a["ws"], a["rows"], a["cols"], a["x"], a["xd"], a["stride"], a["batch"], a["y"],
                      a["yd"]) == status
    if not {"xd", "stride"} & set(change):
        assert L.mx4_gemm_mx4(None, a["w"], a["ws"], a["rows"], a["cols"], a["x"], a["x"], a["batch"], a["y"],
                              a["yd"]) == status


CACHES = [({"head_dim": 96}, UNSUPPORTED), ({"page_tokens": 0}, INVALID), ({"page_tokens": 40}, INVALID),
          ({"page_tokens": 8192}, INVALID), ({"pages": 0}, INVALID), ({"kv_heads": 0}, INVALID),
          ({"kv_heads": 2000}, INVALID)]
ROWS = [({"data": 0}, INVALID), ({"data": P + 16}, INVALID), ({"rows": 0}, OK), ({"batch": 0}, INVALID),
        ({"batch": 70000}, INVALID), ({"rows": 5}, INVALID), ({"rows": 1 << 30}, INVALID), ({"lens": 0}, INVALID),
        ({"lens": P + 2}, INVALID), ({"page_table": 0}, INVALID), ({"page_table": P + 1}, INVALID),
        ({"starts": P + 2}, INVALID), ({"table_stride": -1}, INVALID), ({"table_width": 1 << 26}, INVALID)]
TIMES = [({"q_heads": 0}, INVALID), ({"q_heads": 3}, INVALID), ({"window": 1 << 31}, INVALID),
         ({"sinks": 1 << 31}, INVALID), ({"scale": float("inf")}, INVALID), ({"scale": float("nan")}, INVALID)]


def _cache(change):
    a = {"data": P, "pages": 4, "kv_heads": 2, "head_dim": 64, "page_tokens": 64}
    a.update({k: v for k, v in change.items() if k in a})
    return mx4._Cache(*a.values())


def _rows(change):
    a = {"page_table": P, "table_stride": 4, "lens": P, "starts": 0, "batch": 2, "table_width": 4, "rows": 2}
    a.update({k: v for k, v in change.items() if k in a})
    return mx4._Rows(*a.values())


def _attention(change):
    a = {"q_heads": 4, "max_rows": 0, "max_len": 0, "window": 0, "sinks": 0, "scale": 1.0}
    a.update({k: v for k, v in change.items() if k in a})
    return mx4._Attention(*a.values())


@pytest.mark.parametrize("change,status", CACHES)
def test_cache_shapes(L, change, status):
    n = ctypes.c_size_t(0)
    assert L.kv4_bytes(_cache(change), n) == status
    assert L.kv4_bytes(_cache({}), None) == INVALID
    assert L.kv4_bytes(None, n) == INVALID


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_cache_bytes_are_4_25_bits_per_element(L, head_dim):
    n = ctypes.c_size_t(0)
    assert L.kv4_bytes(_cache({"head_dim": head_dim}), n) == OK
    assert n.value * 8 == 4 * 2 * 64 * 2 * head_dim * 4.25


@pytest.mark.parametrize("change,status", CACHES + ROWS)
def test_append_and_read(L, change, status):
    strides = (ctypes.c_int64 * 4)(128, 64, 128, 64)
    c, r = _cache(change), _rows(change)
    assert L.kv4_append(None, c, r, P, P, ecw.DT_BF16, strides) == status
    assert L.kv4_read(None, c, r, P, P, ecw.DT_BF16) == status


def test_append_and_read_operands(L):
    strides = (ctypes.c_int64 * 4)(128, 64, 128, 64)
    c, r = _cache({}), _rows({})
    for k, v, dt, st in ((0, P, ecw.DT_BF16, strides), (P, P + 1, ecw.DT_BF16, strides), (P, P, ecw.DT_I8, strides),
                         (P, P, ecw.DT_BF16, None), (P, P + 2, ecw.DT_F32, strides),
                         (P, P, ecw.DT_F16, (ctypes.c_int64 * 4)(128, 64, -128, 64))):
        assert L.kv4_append(None, c, r, k, v, dt, st) == INVALID
    for k, v, dt in ((0, P, ecw.DT_BF16), (P, P + 8, ecw.DT_BF16), (P, P, ecw.DT_I8)):
        assert L.kv4_read(None, c, r, k, v, dt) == INVALID
    assert L.kv4_append(None, c, None, P, P, ecw.DT_BF16, strides) == INVALID


@pytest.mark.parametrize("change,status", CACHES + ROWS + TIMES)
def test_attend(L, change, status):
    n = ctypes.c_size_t(0)
    c, r, a = _cache(change), _rows(change), _attention(change)
    assert L.kv4_attend_workspace_size(c, r, a, n) == status
    assert L.kv4_attend(None, c, r, a, P, ecw.DT_BF16, 256, 64, P, P, 1 << 30) == status


def test_attend_operands_and_workspace(L):
    n = ctypes.c_size_t(0)
    c, r, a = _cache({}), _rows({"table_width": 4096}), _attention({})
    assert L.kv4_attend_workspace_size(c, r, a, n) == OK and n.value > 0
    for q, dt, row, head, o, ws, size in (
            (0, ecw.DT_BF16, 256, 64, P, P, n.value), (P + 1, ecw.DT_BF16, 256, 64, P, P, n.value),
            (P, ecw.DT_F32, 256, 64, P, P, n.value), (P, ecw.DT_BF16, -1, 64, P, P, n.value),
            (P, ecw.DT_BF16, 256, 64, 0, P, n.value), (P, ecw.DT_BF16, 256, 64, P + 8, P, n.value),
            (P, ecw.DT_BF16, 256, 64, P, 0, n.value), (P, ecw.DT_BF16, 256, 64, P, P + 4, n.value),
            (P, ecw.DT_BF16, 256, 64, P, P, n.value - 1)):
        assert L.kv4_attend(None, c, r, a, q, dt, row, head, o, ws, size) == INVALID
    assert L.kv4_attend(None, c, r, None, P, ecw.DT_BF16, 256, 64, P, P, n.value) == INVALID


def test_tensors_off_the_gpu_are_refused():
    with pytest.raises(TypeError):
        ecw.mx4_quantize(torch.zeros(2, 64))
    with pytest.raises(TypeError):
        ecw.MX4Tensor(torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8), 2, 128)
    with pytest.raises(ValueError):
        ecw.KV4Cache(0, 1, 64)


def test_scale_that_log2_e_takes_past_the_range(L):
    """Scores are taken to base 2: scale * log2(e) has to be a number too."""
    n = ctypes.c_size_t(0)
    for scale, status in ((2.3e38, OK), (-2.3e38, OK), (2.5e38, INVALID), (-3.4e38, INVALID)):
        assert L.kv4_attend_workspace_size(_cache({}), _rows({}), _attention({"scale": scale}), n) == status


def test_launches_past_2_32_threads_are_refused_by_name(L):
    """A launch has fewer than 2^32 threads along its grid; one that would need more says so
    and does not reach the driver."""
    rows, cols = 1 << 22, 1 << 13  # 2^32 lanes of 8 elements
    assert L.mx4_quantize(None, P, ecw.DT_BF16, cols, rows, cols, P, P) == UNSUPPORTED
    assert L.mx4_dequantize(None, P, P, rows, cols, P, ecw.DT_BF16) == UNSUPPORTED
    strides = (ctypes.c_int64 * 4)(128, 64, 128, 64)
    c, r = _cache({"kv_heads": 1024, "head_dim": 256}), _rows({"rows": 1 << 18, "batch": 1})
    assert L.kv4_append(None, c, r, P, P, ecw.DT_BF16, strides) == UNSUPPORTED
    assert L.kv4_read(None, c, r, P, P, ecw.DT_BF16) == UNSUPPORTED
    assert L.mx4_gemm(None, P, P, 1 << 20, 7, P, ecw.DT_BF16, 8, 1 << 12, P, ecw.DT_F32) == UNSUPPORTED  # an output a lane
    assert L.mx4_gemm(None, P, P, 1 << 30, 64, P, ecw.DT_BF16, 64, 1, P, ecw.DT_F32) == UNSUPPORTED     # 16 rows a block
    assert L.mx4_gemm(None, P, P, 1 << 30, 64, P, ecw.DT_BF16, 64, 1 << 12, P, ecw.DT_F32) == UNSUPPORTED
    assert L.mx4_gemm_mx4(None, P, P, 1 << 30, 64, P, P, 1 << 20, P, ecw.DT_F32) == UNSUPPORTED


def test_attention_of_very_many_rows_is_not_split(L):
    """The join of splits takes 64 threads for each row and head: hints of short sequences do
    not have it launched for more of them than a grid holds."""
    n = ctypes.c_size_t(0)
    a = {"max_rows": 1, "q_heads": 16, "kv_heads": 2, "table_width": 4096, "starts": P, "batch": 1}
    for rows, split in ((1 << 20, True), (1 << 22, False)):
        c, r, t = _cache(a), _rows({**a, "rows": rows}), _attention(a)
        assert L.kv4_attend_workspace_size(c, r, t, n) == OK and (n.value > 0) == split


def test_build_without_python_headers_still_gives_the_library(monkeypatch, tmp_path, capsys):
    """libecw.so needs neither Python's headers nor torch's; without them only the binding of
    the 4-bit calls is left out, with a word."""
    from entropy_coded_weight_amd import build
    ran, bind, paths = [], tmp_path / "_mx4.so", sysconfig.get_paths()
    bind.write_text("of an older build")
    monkeypatch.setattr(build, "BIND", str(bind))
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: ran.append(cmd))
    monkeypatch.setattr(os, "replace", lambda a, b: ran.append([a, b]))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {**paths, "include": str(tmp_path)})
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libecw.so"))
    assert build.build() == build.LIB
    assert [build.LIB + ".tmp", build.LIB] in ran and not any("mx4_bind.cpp" in part for cmd in ran for part in cmd)
    assert not bind.exists() and "Python.h" in capsys.readouterr().err
