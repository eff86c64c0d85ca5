"""The 4-bit key/value cache on the GPU: append and read bit for bit, attention against
its float64 definition.

Tolerance of attention, per output: every weight is rounded to bf16 before the second
product (half a step, 2^-8 of each: 2^-8 sum p |v| in all) and carries the error of its
score, which the normalisation can double: a score's sum of D products in fp32, one
rounding of 2^-23 of sum |q k| for each of the D / 32 instructions and the 64 additions
inside, and 2^-18 for the exponential's argument and result (scores here stay under
2^5, half an fp32 step of 2^-19 there).  The sums over tokens add 2^-23 for each of
the T / 32 tiles and 128 more.  Then half a step of the output type."""
import threading
from types import SimpleNamespace

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
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def _say(*a):
    print("[gpu]", *a, flush=True)


def _normal(seed, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


class Bed:
    """A cache full of rubbish (NaN scales), sequences of given lengths appended to it."""

    def __init__(self, lens, heads, dim, page=64, dtype=BF16, spare=3, seed=0, gone=(), k=None, v=None):
        self.lens, self.heads, self.dim, self.page = list(lens), heads, dim, page
        width = max(1, -(-max([*lens, 1]) // page))
        pages = sum(-(-n // page) for n in lens) + spare
        self.cache = ecw.KV4Cache(pages, heads, dim, page_tokens=page)
        self.cache.data.fill_(255)
        order = np.random.default_rng(seed).permutation(pages)
        table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                table[b, i] = order[at]
                at += 1
        for b, i in gone:
            table[b, i] = -1 if i % 2 else pages  # both sides of the range
        self.table = torch.from_numpy(table).cuda()
        self.k = [k[b] if k else _normal(seed + 10 + b, n, heads, dim, dtype=dtype) for b, n in enumerate(lens)]
        self.v = [v[b] if v else _normal(seed + 50 + b, n, heads, dim, dtype=dtype) for b, n in enumerate(lens)]
        starts = np.concatenate([[0], np.cumsum(lens)])
        if starts[-1]:
            self.cache.append(torch.cat(self.k), torch.cat(self.v), self.table, I32(lens), starts=I32(starts.tolist()))
        self.there = []
        for b, n in enumerate(lens):
            p = table[b][np.arange(n) // page]
            self.there.append((p >= 0) & (p < pages))

    def check(self, o, q, rows, window=0, sinks=0, scale=None, lens=None, skip=(), grid=1e-30):
        """rows: how many of each sequence, in order."""
        scale = self.dim ** -0.5 if scale is None else scale
        half = {BF16: 2.0 ** -8, FP16: 2.0 ** -11}[o.dtype]
        got, qd, at = F64(o), F64(q), 0
        for b, n in enumerate(rows):
            length = (lens or self.lens)[b]
            want, mag, dot = R.attend_rows(qd[at:at + n], np.arange(length - n, length), R.rounded(F64(self.k[b])),
                                           R.rounded(F64(self.v[b])), self.there[b], scale, window, sinks)
            score = (self.dim / 32 + 64) * 2.0 ** -23 * dot + 2.0 ** -18
            tol = (2.0 ** -8 + 2 * score + (len(self.k[b]) / 32 + 128) * 2.0 ** -23) * mag
            tol = tol + half * (np.abs(want) + tol) + grid
            mine = got[at:at + n]
            if b not in skip:
                nan = np.isnan(want)
                assert np.array_equal(nan, np.isnan(mine)), f"sequence {b}: NaN elsewhere"
                err = np.abs(mine - want)
                assert (err[~nan] <= tol[~nan]).all(), f"sequence {b}: worst {np.nanmax(err / tol)}"
            at += n
        return got[at:]


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("page", [32, 64, 96])
def test_append_and_read_back(dim, dtype, page):
    _say("append", dim, dtype, page)
    lens = [1, 0, page, 2 * page + 7, 31]
    bed = Bed(lens, 3, dim, page, dtype)
    starts = I32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    for out in (BF16, FP32, FP16):
        k, v = bed.cache.read(bed.table, I32(lens), sum(lens), starts=starts, dtype=out)
        for got, want in ((k, bed.k), (v, bed.v)):
            assert torch.equal(got.cpu(), torch.from_numpy(R.rounded(F64(torch.cat(want)))).to(out))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_touches_only_its_tokens(dim):
    _say("append alone", dim)
    bed = Bed([70, 40], 2, dim)
    k, v = _normal(1, 2, 2, dim), _normal(2, 2, 2, dim)
    bed.cache.append(k, v, bed.table, I32([50, 33]))  # one row each: tokens 49 and 32
    got_k, got_v = bed.cache.read(bed.table, I32([70, 40]), 110, starts=I32([0, 70, 110]))
    for got, old, new in ((got_k, bed.k, k), (got_v, bed.v, v)):
        want = R.rounded(F64(torch.cat(old)))
        want[49], want[70 + 32] = R.rounded(F64(new))
        assert np.array_equal(F64(got), want)
    whole = bed.cache.data.cpu()
    used = torch.zeros(bed.cache.pages, dtype=torch.bool)
    used[bed.table[bed.table >= 0].long().cpu()] = True
    assert bool((whole.view(bed.cache.pages, -1)[~used] == 255).all()), "a page of nobody was written"


def test_append_strides_and_several_rows():
    _say("append strided")
    big = _normal(3, 12, 7, 200, dtype=FP16)
    for off in (0, 1, 8):
        k, v = big[:, 1:3, off:off + 128], big.transpose(0, 0)[:, 4:6, off + 5:off + 133]
        bed = Bed([64, 200, 10], 2, 128)
        bed.cache.append(k, v, bed.table, I32([64, 104, 10]))  # four rows each
        got = bed.cache.read(bed.table, I32([64, 104, 10]), 12)
        assert np.array_equal(F64(got[0]), R.rounded(F64(k))) and np.array_equal(F64(got[1]), R.rounded(F64(v)))


def test_rows_without_a_page_are_dropped():
    _say("append nowhere")
    cache = ecw.KV4Cache(4, 1, 64, page_tokens=32)
    cache.data.fill_(7)
    k = torch.ones(6, 1, 64, device="cuda")
    table = I32([[-1, 9], [4, 2 ** 31 - 1], [-2 ** 31, -5], [0, 1], [0, 1], [0, 1]])
    lens = I32([5, 40, 33, 0, -7, 1000])  # unmapped; no token; past the table's end
    cache.append(k, k, table, lens)
    assert bool((cache.data == 7).all())
    for t in cache.read(table, lens, 6):
        assert not t.any()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 16), (2, 17)])
def test_one_row_each(heads, group, dim, dtype):
    _say("attend", heads, group, dim, dtype)
    bed = Bed([1, 31, 32, 33, 64, 65, 300, 1027], heads, dim, dtype=dtype)
    q = _normal(99, 8, heads * group, dim, dtype=dtype, scale=1.5)
    o = bed.cache.attend(q, bed.table, I32(bed.lens))
    bed.check(o, q, [1] * 8)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (17, 0), (32, 4), (100, 40), (5000, 4), (64, 2000)])
@pytest.mark.parametrize("dim,rows", [(128, [3, 1, 33, 40, 7]), (64, [20, 1, 33, 0, 70]), (256, [5, 1, 17, 40, 2])])
def test_windows_sinks_and_ragged_rows(dim, rows, window, sinks, dtype):
    _say("attend window", dim, rows, window, sinks, dtype)
    bed = Bed([50, 1, 33, 40, 700], 2, dim, dtype=dtype)
    starts = np.concatenate([[0], np.cumsum(rows)])
    q = _normal(98, sum(rows), 6, dim, dtype=dtype)
    for hints in ({}, {"max_rows": 70, "max_len": 700}, {"max_rows": 1, "max_len": 1}):
        o = bed.cache.attend(q, bed.table, I32(bed.lens), starts=I32(starts.tolist()), window=window, sinks=sinks, **hints)
        bed.check(o, q, rows, window, sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 4, 200])
def test_long_sequences_are_split_and_joined(dim, n):
    _say("attend long", dim, n)
    bed = Bed([5000, 3111], 2, dim)
    q = _normal(97, 2 * n, 4, dim, scale=2.0)
    bed.check(bed.cache.attend(q, bed.table, I32(bed.lens)), q, [n, n])
    bed.check(bed.cache.attend(q, bed.table, I32(bed.lens), window=1000, sinks=9), q, [n, n], 1000, 9)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,rows", [([36000], 1), ([36000], 20), ([20000, 40], 2), ([0, 9000], 1), ([3000], 3)])
def test_one_long_sequence(dim, lens, rows):
    """As many splits as there are, and their number on both sides of 64 and of a wave's share."""
    _say("attend long", dim, lens, rows)
    bed = Bed(lens, 1, dim)
    q = _normal(83, rows * len(lens), 2, dim)
    bed.check(bed.cache.attend(q, bed.table, I32(lens)), q, [rows] * len(lens))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,group,rows", [(64, 8, [23, 1, 70, 0, 300]), (128, 4, [500, 3, 49, 1, 200]),
                                            (128, 1, [700, 600, 190, 1, 255]), (64, 1, [256, 257, 31, 33, 512])])
def test_many_rows(dim, group, rows, dtype):
    _say("attend many", dim, group, rows, dtype)
    lens = [n + extra for n, extra in zip(rows, (0, 900, 31, 5, 700))]
    bed = Bed(lens, 2, dim, dtype=dtype, gone=[(4, 3), (4, 4), (4, 5)])
    starts = np.concatenate([[0], np.cumsum(rows)])
    q = _normal(82, sum(rows) + 3, 2 * group, dim, dtype=dtype)  # three rows of nobody
    for window, sinks in ((0, 0), (70, 33)):
        o = bed.cache.attend(q, bed.table, I32(lens), starts=I32(starts.tolist()), max_rows=700, window=window,
                             sinks=sinks)
        rest = bed.check(o, q, rows, window, sinks)
        assert not rest.any()


@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_and_bad_values(dim):
    _say("attend many NaN", dim)
    k, v = [_normal(1, 500, 1, dim)], [_normal(2, 500, 1, dim)]
    v[0][433, 0, 40] = float("nan")
    v[0][460, 0, 3] = float("inf")
    k[0][480, 0, 0] = float("nan")
    bed = Bed([500], 1, dim, k=k, v=v)
    q = _normal(81, 300, 1, dim)
    bed.check(bed.cache.attend(q, bed.table, I32([500])), q, [300])
    bed.check(bed.cache.attend(q, bed.table, I32([500]), window=20), q, [300], 20)


@pytest.mark.parametrize("page", [32, 96, 128, 416, 4096])
@pytest.mark.parametrize("n", [1, 20])
def test_page_sizes(page, n):
    _say("attend pages", page, n)
    bed = Bed([37, 900, 1300], 1, 64, page=page)
    q = _normal(83, 3 * n, 3, 64)
    for window, sinks in ((0, 0), (300, 5)):
        bed.check(bed.cache.attend(q, bed.table, I32(bed.lens), window=window, sinks=sinks), q, [n] * 3, window, sinks)


@pytest.mark.parametrize("n", [1, 6, 40])
def test_missing_pages_and_rows_that_see_nothing(n):
    _say("attend missing", n)
    bed = Bed([300, 64, 500], 2, 128, gone=[(0, 0), (0, 3), (1, 0), (2, 5), (2, 6), (2, 7)])
    q = _normal(96, 3 * n, 4, 128)
    for window, sinks in ((0, 0), (60, 3), (200, 70)):
        o = bed.cache.attend(q, bed.table, I32(bed.lens), window=window, sinks=sinks)
        bed.check(o, q, [n] * 3, window, sinks)
        assert not o[n:2 * n].any()


def test_no_tokens_and_rows_of_no_sequence():
    _say("attend empty")
    bed = Bed([40, 0, 90], 2, 64)
    q = _normal(95, 12, 2, 64)
    starts = I32([2, 4, 5, 9])  # rows 0, 1 and 9..11 belong to nobody; the second sequence has no token
    for out in (None, torch.full_like(q, 5.0)):
        o = bed.cache.attend(q, bed.table, I32(bed.lens), starts=starts, out=out)
        assert not o[:2].any() and not o[9:].any() and not o[4:5].any()
        bed.check(o[2:9], q[2:9], [2, 1, 4], skip=(1,))
    none = bed.cache.attend(q, bed.table, I32([0, -3, -2 ** 31]))
    assert not none.any()
    wide = bed.cache.attend(q[:3], bed.table[:, :0], I32(bed.lens))  # a table of no pages
    assert not wide.any()
    assert bed.cache.attend(q[:0], bed.table, I32(bed.lens)).shape == (0, 2, 64)


def test_more_rows_than_tokens():
    """Rows before a sequence's beginning see nothing."""
    _say("attend short")
    bed = Bed([3], 1, 64)
    q = _normal(94, 8, 1, 64)
    o = bed.cache.attend(q, bed.table, I32([3]))
    assert not o[:5].any()
    bed.check(o[5:], q[5:], [3])


def test_lengths_past_the_table():
    _say("attend past the table")
    bed = Bed([128], 1, 64)
    q = _normal(93, 1, 2, 64)
    o = bed.cache.attend(q, bed.table, I32([4000]))
    bed.check(o, q, [1])
    for big in (2 ** 31 - 1, 2 ** 30):
        bed.check(bed.cache.attend(q, bed.table, I32([big])), q, [1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 9, 40])
def test_nan_and_infinity_reach_only_rows_that_see_them(dim, n):
    _say("attend NaN", dim, n)
    k, v = [_normal(1, 400, 2, dim)], [_normal(2, 400, 2, dim)]
    v[0][391, 0, 40] = float("nan")     # visible to the rows at or behind it
    v[0][20, 1, 5] = float("inf")       # outside the window
    k[0][10, 0, 0] = float("nan")
    k[0][395, 1, 3] = float("inf")
    bed = Bed([400], 2, dim, k=k, v=v)
    q = _normal(92, n, 4, dim)
    bed.check(bed.cache.attend(q, bed.table, I32([400]), window=100), q, [n], 100)
    bed.check(bed.cache.attend(q, bed.table, I32([400])), q, [n])


@pytest.mark.parametrize("n", [1, 20])
def test_fp16_queries_over_values_of_other_types(n):
    """Small values round to fp16's grid (by 2^-25 at most); values past its range are NaN
    to the rows that see them, and to no other."""
    _say("attend fp16 range", n)
    k, v = [_normal(1, 200, 1, 64)], [_normal(2, 200, 1, 64)]
    v[0][:, :, :32] *= 2.0 ** -30
    k[0][50:60, :, 32:] *= 2.0 ** -28
    bed = Bed([200], 1, 64, k=k, v=v)
    q = _normal(92, n, 2, 64, dtype=FP16)
    o = bed.cache.attend(q, bed.table, I32([200]))
    bed.check(o, q, [n], grid=2.0 ** -24)  # the values' and the output's
    v[0][190, 0, 3] = 1e6
    bed = Bed([200], 1, 64, k=k, v=v)
    o = bed.cache.attend(q, bed.table, I32([200]))
    sees = torch.arange(200 - n, 200) >= 190
    assert bool(torch.isnan(o[sees][..., :32]).all()) and bool(torch.isfinite(o[sees][..., 32:]).all())
    assert bool(torch.isfinite(o[~sees]).all())


def test_peaked_and_equal_scores():
    _say("attend peaked")
    k, v = [torch.zeros(500, 1, 128, dtype=BF16, device="cuda")], [_normal(2, 500, 1, 128)]
    q = _normal(91, 2, 2, 128)
    bed = Bed([500], 1, 128, k=k, v=v)
    bed.check(bed.cache.attend(q, bed.table, I32([500])), q, [2])
    k[0][250] = 4.0
    q[:] = 1.0
    bed = Bed([500], 1, 128, k=k, v=v)
    bed.check(bed.cache.attend(q, bed.table, I32([500])), q, [2])
    minus = torch.full_like(q, -1.0)
    bed.check(bed.cache.attend(minus, bed.table, I32([500])), minus, [2])


def test_scores_of_minus_infinity():
    """All visible scores -inf: NaN, as the definition says, not the zeros of an empty row."""
    _say("attend -inf")
    k, v = [torch.ones(64, 1, 64, dtype=BF16, device="cuda")], [_normal(2, 64, 1, 64)]
    k[0][40:, 0, 0] = -1
    q = torch.ones(1, 1, 64, dtype=BF16, device="cuda")
    q[0, 0, 0] = -float("inf")
    bed = Bed([64], 1, 64, k=k, v=v)
    assert bool(torch.isnan(bed.cache.attend(q, bed.table, I32([40]))).all())


@pytest.mark.parametrize("off,pad", [(0, 0), (1, 3), (8, 8)])
def test_query_strides_and_alignment(off, pad):
    _say("attend strided", off, pad)
    bed = Bed([100, 37], 2, 64, dtype=FP16)
    big = _normal(90, 6, 5, 64 + off + pad, dtype=FP16)
    q = big[:, :4, off:off + 64]
    bed.check(bed.cache.attend(q, bed.table, I32(bed.lens)), q, [3, 3])
    q = big.transpose(0, 1)[:4, :4, off:off + 64]
    bed.check(bed.cache.attend(q, bed.table, I32(bed.lens)), q, [2, 2])


def test_page_tables_at_a_stride_and_scale():
    _say("attend table stride")
    bed = Bed([100, 200], 1, 128)
    wide = torch.full((2, 9), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :bed.table.shape[1]] = bed.table
    q = _normal(89, 2, 2, 128)
    bed.check(bed.cache.attend(q, wide[:, :bed.table.shape[1]], I32(bed.lens), scale=0.31), q, [1, 1], scale=0.31)


def test_cache_offsets_pass_32_bits():
    _say("attend large cache")
    cache = ecw.KV4Cache(70000, 8, 128, page_tokens=64)  # 4.9e9 bytes
    bed = Bed([200], 8, 128)
    table = I32([[69999, 61000, 69998, 3]])
    cache.append(bed.k[0], bed.v[0], table, I32([200]))
    bed.cache, bed.table = cache, table
    q = _normal(88, 2, 16, 128)
    bed.check(cache.attend(q, table, I32([200])), q, [2])
    got = cache.read(table, I32([200]), 200)
    assert np.array_equal(F64(got[0]), R.rounded(F64(bed.k[0])))


def test_another_stream_and_graph_replays():
    _say("attend graph")
    bed = Bed([300, 2000], 2, 128)
    lens = I32(bed.lens)
    q, k, v = _normal(87, 2, 8, 128), _normal(86, 2, 2, 128), _normal(85, 2, 2, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = bed.cache.attend(q, bed.table, lens, stream=s)
    s.synchronize()
    bed.check(o, q, [1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bed.cache.append(k, v, bed.table, lens)
        o = bed.cache.attend(q, bed.table, lens, max_len=2000)
        back = bed.cache.read(bed.table, lens, 2)
    for step in range(4):
        k.copy_(_normal(20 + step, 2, 2, 128))
        q.copy_(_normal(30 + step, 2, 8, 128))
        lens.copy_(I32([300 - step, 2000 - 40 * step]))
        g.replay()
        torch.cuda.synchronize()
        got = o.clone(), back[0].clone()
        bed.cache.append(k, v, bed.table, lens)
        assert torch.equal(got[0], bed.cache.attend(q, bed.table, lens, max_len=2000))
        assert np.array_equal(F64(got[1]), R.rounded(F64(k)))


def test_same_result_every_time():
    bed = Bed([3000, 77], 2, 128)
    q = _normal(84, 2, 8, 128)
    first = bed.cache.attend(q, bed.table, I32(bed.lens))
    for _ in range(5):
        assert torch.equal(bed.cache.attend(q, bed.table, I32(bed.lens)), first)


def test_refusals():
    bed = Bed([40, 40], 2, 64)
    q, lens = _normal(1, 2, 4, 64), I32([40, 40])
    for bad, error in ((q.float(), TypeError), (q[:, :3], ValueError), (q[..., :32], ValueError), (q.cpu(), TypeError),
                       (q[0], ValueError), (q[:1], ValueError), (_normal(1, 2, 64, 4).transpose(1, 2), TypeError)):
        with pytest.raises(error):
            bed.cache.attend(bad, bed.table, lens)
    for kw in ({"window": -1}, {"sinks": -1}, {"max_len": -2}, {"out": torch.empty(2, 4, 32, device="cuda")},
               {"starts": I32([0, 2])}):
        with pytest.raises(ValueError):
            bed.cache.attend(q, bed.table, lens, **kw)
    with pytest.raises(ecw.EcwError):
        bed.cache.attend(q, bed.table, lens, scale=float("nan"))
    with pytest.raises(TypeError):
        bed.cache.attend(q, bed.table.long(), lens)
    with pytest.raises(ValueError):
        bed.cache.attend(q, bed.table, lens[:1])
    k = q[:, :2].contiguous()
    with pytest.raises(ValueError):
        bed.cache.append(k, k[:1], bed.table, lens)
    with pytest.raises(ValueError):
        bed.cache.append(q, q, bed.table, lens)
    with pytest.raises(ValueError):
        bed.cache.append(k, k.half(), bed.table, lens)
    with pytest.raises(TypeError):
        bed.cache.append(k.double(), k.double(), bed.table, lens)
    with pytest.raises(ValueError):
        bed.cache.read(bed.table, lens, 3)
    with pytest.raises(ValueError):
        bed.cache.read(bed.table, lens, -1)
    for args in ((0, 1, 64), (1, 0, 64), (1, 1, 0), (1, 1, 64, -32)):
        with pytest.raises(ValueError):
            ecw.KV4Cache(*args)
    for args in ((1, 1, 96), (1, 1, 64, 48)):
        with pytest.raises(ecw.EcwError):
            ecw.KV4Cache(*args)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("value", [1e6, -1e6, 65536.0])
def test_fp16_queries_over_keys_past_their_range(value, dim, n):
    """A key block past fp16's range is NaN to the rows that see it, whatever the sign and
    size of its product with the query, and nothing to the others; 65504 is in the range."""
    _say("attend fp16 key range", value, dim, n)
    k, v = [_normal(1, 200, 1, dim)], [_normal(2, 200, 1, dim)]
    k[0][190, 0, 3] = value
    k[0][195, 0, dim - 1] = 49152.0  # the largest that fp16 holds in 4 bits
    bed = Bed([200], 1, dim, k=k, v=v)
    bed.k[0] = k[0].clone()
    bed.k[0][190, 0, :32] = float("nan")
    q = _normal(92, n, 2, dim, dtype=FP16)
    q[:, :, 3] = 1e-4
    q[:, :, dim - 1] = 1e-4
    bed.check(bed.cache.attend(q, bed.table, I32([200])), q, [n])
    bed.check(bed.cache.attend(q, bed.table, I32([200]), window=6), q, [n], 6)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n", [1, 20])
def test_a_visible_nan_value_of_no_weight_is_nan_in_every_split(n, dtype):
    """A weight may be too small for any number, but 0 times NaN is NaN, in whichever split
    of the tokens the value lies."""
    _say("attend NaN of no weight", n, dtype)
    k = [torch.full((5000, 1, 64), -6.0, dtype=BF16, device="cuda")]
    v = [_normal(2, 5000, 1, 64)]
    k[0][4000] = 6.0
    v[0][5, 0, 40] = float("nan")
    bed = Bed([5000], 1, 64, k=k, v=v)
    q = torch.full((n, 2, 64), 8.0, dtype=dtype, device="cuda")  # scores of 384 and -384
    for hints in ({}, {"max_len": 1}, {"max_len": 1000}, {"max_len": 5000}):
        bed.check(bed.cache.attend(q, bed.table, I32([5000]), **hints), q, [n])
    bed.check(bed.cache.attend(q, bed.table, I32([5000]), window=4000), q, [n], 4000)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 20])
def test_values_near_the_end_of_the_range(dim, n):
    """bf16 values up to 2^127: an average of them is one of them, not an infinity."""
    _say("attend large values", dim, n)
    lens = [300, 6000]
    v = [torch.full((m, 1, dim), 2.0 ** 127, dtype=BF16, device="cuda") for m in lens]
    bed = Bed(lens, 1, dim, v=v)
    q = _normal(79, 2 * n, 2, dim, scale=2.0)
    o = bed.cache.attend(q, bed.table, I32(lens))
    bed.check(o, q, [n, n])
    v = [_normal(3, m, 1, dim, scale=2.0 ** -70) for m in lens]  # and small ones keep their bits
    bed = Bed(lens, 1, dim, v=v)
    bed.check(bed.cache.attend(q, bed.table, I32(lens)), q, [n, n], grid=2.0 ** -100)


def test_a_stream_of_another_device_is_refused():
    other = SimpleNamespace(device=torch.device("cuda", 1))  # refused before anything is done with it
    bed = Bed([40], 2, 64)
    q, lens = _normal(1, 1, 4, 64), I32([40])
    k = q[:, :2].contiguous()
    w = ecw.mx4_quantize(_normal(2, 16, 64))
    for call in (lambda: bed.cache.attend(q, bed.table, lens, stream=other),
                 lambda: bed.cache.append(k, k, bed.table, lens, stream=other),
                 lambda: bed.cache.read(bed.table, lens, 1, stream=other),
                 lambda: ecw.mx4_quantize(q[0], stream=other), lambda: w.dequantize(stream=other),
                 lambda: w.gemm(_normal(3, 2, 64), stream=other), lambda: w.gemm(w, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_given_outputs_count_as_written():
    """out= and y= advance the tensors' versions, so that autograd notices if it holds them."""
    x = _normal(1, 4, 64)
    w = ecw.mx4_quantize(x)
    y, d = torch.empty(4, 4, device="cuda"), torch.empty(4, 64, device="cuda")
    bed = Bed([40], 2, 64)
    q, lens = _normal(1, 1, 4, 64), I32([40])
    o = torch.empty_like(q)
    for t, call in ((y, lambda: w.gemm(x, y=y)), (y, lambda: w.gemm(w, y=y)), (d, lambda: w.dequantize(out=d)),
                    (w.codes, lambda: ecw.mx4_quantize(x, out=w)), (w.scales, lambda: ecw.mx4_quantize(x, out=w)),
                    (o, lambda: bed.cache.attend(q, bed.table, lens, out=o)),
                    (bed.cache.data, lambda: bed.cache.append(q[:, :2], q[:, 2:], bed.table, lens))):
        before = t._version
        call()
        assert t._version > before
    with torch.inference_mode():
        inside = torch.empty(4, 4, device="cuda")
    assert torch.equal(w.gemm(x, y=inside), w.gemm(x))  # has no version to advance
    a = torch.ones(1, 4, 64, device="cuda", requires_grad=True)
    held = torch.ones(1, 4, 64, dtype=BF16, device="cuda")
    loss = (a * held).sum()
    bed.cache.attend(q, bed.table, lens, out=held)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("dim,group,n", [(64, 8, 1), (64, 8, 40), (128, 4, 1), (128, 4, 40), (256, 2, 1), (256, 2, 9)])
def test_fp16_weights_are_fp16(dim, group, n):
    """With an fp16 query the softmax weights have fp16's bits: half a step, 2^-11, of each in
    the sum over values and in the weights' own sum, and fp16's smallest step, 2^-25 against
    a largest weight of 2^7 or more, of each token.  The other terms as in Bed.check."""
    _say("attend fp16 weights", dim, group, n)
    bed = Bed([1027, 60], 2, dim, dtype=FP16)
    q = _normal(78, 2 * n, 2 * group, dim, dtype=FP16, scale=1.5)
    got, qd = F64(bed.cache.attend(q, bed.table, I32(bed.lens))), F64(q)
    for b, length in enumerate(bed.lens):
        kv, vv = R.rounded(F64(bed.k[b])), R.rounded(F64(bed.v[b]))
        want, mag, dot = R.attend_rows(qd[b * n:b * n + n], np.arange(length - n, length), kv, vv, bed.there[b],
                                       dim ** -0.5, 0, 0)
        score = (dim / 32 + 64) * 2.0 ** -23 * dot + 2.0 ** -18
        tol = (2 * 2.0 ** -11 + 2 * score + (length / 32 + 128) * 2.0 ** -23) * mag + 2 * length * 2.0 ** -32 * np.abs(vv).max()
        tol = tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
        err = np.abs(got[b * n:b * n + n] - want)
        assert (err <= tol).all(), f"sequence {b}: worst {(err / tol).max()}"


def test_graph_replays_append_keys_and_values():
    _say("append graph")
    bed = Bed([300, 77], 2, 128)
    lens, k, v = I32(bed.lens), _normal(86, 2, 2, 128), _normal(85, 2, 2, 128)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lens -= 1
        bed.cache.append(k, v, bed.table, lens)
        back = bed.cache.read(bed.table, lens, 2)
    kept = [], []
    for step in range(4):
        k.copy_(_normal(20 + step, 2, 2, 128))
        v.copy_(_normal(40 + step, 2, 2, 128))
        g.replay()
        torch.cuda.synchronize()
        for got, new, rows in zip(back, (k, v), kept):
            rows.insert(0, R.rounded(F64(new)))
            assert np.array_equal(F64(got), rows[0])
    tail = bed.cache.read(bed.table, I32(bed.lens), 10)  # the last five: four new ones and the old last
    for got, old, rows in zip(tail, (bed.k, bed.v), kept):
        for b in range(2):
            want = [*(r[b] for r in rows), R.rounded(F64(old[b][-1]))]
            assert np.array_equal(F64(got).reshape(2, 5, 2, 128)[b], np.stack(want))


def test_two_streams_and_two_threads_at_once():
    """Calls share nothing: a thread each with its stream and cache gives what it gives alone."""
    _say("attend two threads")
    beds = [Bed([5000, 300], 2, 128, seed=s) for s in (0, 1)]
    qs = [_normal(70 + s, 2, 8, 128) for s in (0, 1)]
    alone = [b.cache.attend(q, b.table, I32(b.lens)) for b, q in zip(beds, qs)]
    lens = [I32(b.lens) for b in beds]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i].append(beds[i].cache.attend(qs[i], beds[i].table, lens[i]))
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (0, 1):
        assert len(got[i]) == 20 and all(torch.equal(o, alone[i]) for o in got[i])
