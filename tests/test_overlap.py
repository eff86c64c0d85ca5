"""Whether two strided tensors share a byte (csrc/overlap.h, which the bindings refuse outputs
by), against the sets of bytes themselves."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "entropy_coded_weight_amd", "csrc")
SHIM = """
#include "overlap.h"
extern "C" int meet(const void* a, int64_t ea, int64_t na, const int64_t* sa, const int64_t* ta,
                    const void* b, int64_t eb, int64_t nb, const int64_t* sb, const int64_t* tb) {
  return ecw::boxes_meet(ecw::box_of(a, ea, sa, ta, na), ecw::box_of(b, eb, sb, tb, nb));
}
extern "C" int folded(int64_t e, int64_t n, const int64_t* s, const int64_t* t) { return ecw::box_of(nullptr, e, s, t, n).folded; }
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(d / "shim.cpp"),
                    "-o", str(d / "shim.so")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


def _ints(v):
    return (ctypes.c_int64 * len(v))(*v)


def _args(t):
    return ctypes.c_int64(t.element_size()), ctypes.c_int64(t.dim()), _ints(t.shape), _ints(t.stride())


def _meet(shim, a, b):
    got = [shim.meet(ctypes.c_void_p(x.data_ptr()), *_args(x), ctypes.c_void_p(y.data_ptr()), *_args(y)) for x, y in ((a, b), (b, a))]
    assert got[0] == got[1]
    return bool(got[0])


def _bytes(t):
    at = torch.zeros(1, dtype=torch.int64)
    for n, s in zip(t.shape, t.stride()):
        at = (at[:, None] + torch.arange(n) * s * t.element_size()).flatten()
    return [t.data_ptr() + i + j for i in at.tolist() for j in range(t.element_size())]


def test_views_of_one_buffer(shim):
    wide = torch.zeros(6, 40)
    qkv = torch.zeros(7, 8 * 16)
    heads = qkv.view(7, 8, 16)
    for a, b, want in [
            (wide[:-1, :10], wide[1:, :10], True), (wide[:, :10], wide[:, 10:20], False), (wide[:, :10], wide[:, 9:19], True),
            (wide[:, 30:], wide[:, :10], False), (wide[::2], wide[1::2], False), (wide[:3], wide[3:], False), (wide[:4], wide[3:], True),
            (wide[:-1, 30:], wide[1:, :10], False), (heads[:, :4], heads[:, 4:6], False), (heads[:, :4], heads[:, 1:5], True),
            (heads[..., :8], heads[..., 8:], False), (heads[:, ::2], heads[:, 1::2], False), (heads[:, ::2, 4:], heads[:, ::2, :4], False),
            (heads[:-1, 4:], heads[1:, :4], False), (heads.transpose(0, 1)[:3], heads[:, 3:], False),
            (heads.transpose(0, 1)[:3], heads[:, 2:], True), (wide[2, 5:9], wide[:, 9:30], False), (wide[2, 5:9], wide[:, 8:30], True),
            (wide[0:1].expand(5, 40), wide[1:], False), (wide[0:1].expand(5, 40), wide, True), (wide[:0], wide, False),
            (wide[:, 3:3], wide, False), (wide.view(torch.uint8)[1:3], wide[2:], True), (wide.view(torch.uint8)[1:3], wide[3:], False)]:
        assert bool(set(_bytes(a)) & set(_bytes(b))) == want
        assert _meet(shim, a, b) == want


def test_random_views(shim):
    rng, met = random.Random(1), [0, 0]
    store = torch.zeros(8192, dtype=torch.uint8)

    def view():
        dtype = rng.choice([torch.uint8, torch.bfloat16, torch.float32])
        base = store.view(dtype)
        shape = [rng.randint(1, 5) for _ in range(rng.randint(1, 3))] + [rng.randint(1, 9)]
        strides = [rng.choice([0, 3, 8, 8, 16, 24, 32, 40, 64, 96, 128]) for _ in shape[:-1]] + [1]
        if rng.random() < 0.3:
            strides[-1] = 2
        last = sum((n - 1) * s for n, s in zip(shape, strides))
        return torch.as_strided(base, shape, strides, rng.randint(0, max(0, min(base.numel() - last - 1, 160 // base.element_size()))))

    for _ in range(4000):
        a, b = view(), view()
        want = bool(set(_bytes(a)) & set(_bytes(b)))
        met[want] += 1
        assert _meet(shim, a, b) == want, (a.shape, a.stride(), a.dtype, b.shape, b.stride(), b.dtype, a.data_ptr() - b.data_ptr())
    assert min(met) > 500


def test_views_that_overlap_themselves(shim):
    x = torch.zeros(4000)
    for shape, strides, want in [((4, 6), (6, 1), False), ((4, 6), (5, 1), True), ((3, 2, 8), (16, 8, 1), False), ((3, 2, 8), (8, 24, 1), False),
                                 ((3, 2, 8), (8, 16, 1), True), ((3, 1, 8), (8, 0, 1), False), ((3, 2, 8), (16, 0, 1), True),
                                 ((3, 2, 8), (100, 9, 1), False), ((3, 2, 8), (100, 7, 1), True), ((1, 1, 1), (0, 0, 0), False)]:
        t = torch.as_strided(x, shape, strides)
        assert want == (len(set(_bytes(t))) < len(_bytes(t)))
        assert bool(shim.folded(*_args(t))) == want


def test_many_rows_take_few_steps(shim):
    """Rows of a matrix of any length next to each other's columns: told apart exactly, not by giving up."""
    x = torch.empty(100000, 64)
    assert not _meet(shim, x[:, :32], x[:, 32:]) and _meet(shim, x[:, :33], x[:, 32:]) and _meet(shim, x[:60000, :3], x[50000:, 2:9])
    assert not _meet(shim, x[70000, 5:9], x[:, 9:]) and not _meet(shim, x[::2, :], x[1::2, :])
