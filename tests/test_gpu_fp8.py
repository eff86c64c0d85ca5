"""The 8-bit matrices against their definition in float64: quantisation byte for byte, the
gate within a bracket, products of small whole numbers exactly and others within the
rounding of their sums."""
import numpy as np
import pytest
import torch

import entropy_coded_weight_amd as ecw
from tests import fp8_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(autouse=True)
def _named(request):
    print(f"[gpu] {request.node.name}", flush=True)


def _randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _same_bytes(t, x):
    """FP8Tensor t holds what x [rows, cols] float64 stands for, to the byte."""
    codes, scales = R.quantise(x)
    got, blocks = t.scales.cpu().numpy(), scales.shape[1]
    assert np.array_equal(got[:, :blocks], scales)
    assert (got[:, blocks:] == 127).all()
    assert np.array_equal(t.codes.cpu().numpy(), codes)


# ------------------------------------------------------------------ quantise
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 127), (3, 128), (5, 129), (2, 131), (1, 255), (7, 2049), (33, 333), (2, 16390)])
def test_quantise_bytes(dtype, rows, cols):
    x = _randn(rows, cols, seed=cols) * torch.exp2(4 * _randn(rows, 1, seed=1))
    x[:, ::7] *= 30
    x = x.to(dtype).cuda()
    t = ecw.fp8_quantize(x)
    assert t.shape == (rows, cols) and t.codes.shape == (rows, -(-cols // 128) * 128)
    _same_bytes(t, _f64(x))
    for out in DTYPES:
        with np.errstate(over="ignore"):
            want = torch.from_numpy(R.rounded(_f64(x))).to(out)
        assert torch.equal(t.dequantize(out).cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantise_ties_and_every_level(dtype):
    """Every middle between two levels and its neighbours in the type, beside a 448 that sets
    the scale."""
    u = np.concatenate([R.MIDDLES, R.LEVELS, [448.0]])
    x = torch.from_numpy(np.concatenate([u, -u])).to(dtype)
    x = torch.cat([x, torch.nextafter(x, torch.full_like(x, 1000.0)).clamp(-448, 448),
                   torch.nextafter(x, torch.full_like(x, -1000.0)).clamp(-448, 448)])
    rows = torch.zeros(-(-len(x) // 127), 128, dtype=dtype)
    rows[:, 0] = 448
    for i in range(rows.shape[0]):
        part = x[i * 127:(i + 1) * 127]
        rows[i, 1:1 + len(part)] = part
    for s in (1.0, 2.0 ** -5, 2.0 ** 6):
        y = (rows.double() * s).to(dtype)
        _same_bytes(ecw.fp8_quantize(y.cuda()), y.double().numpy())


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantise_special_blocks(dtype):
    """Zeros, the ends of the range, subnormals, infinities and NaN, each in a block of its
    own: the others are not touched."""
    info = torch.finfo(dtype)
    x = _randn(2, 11 * 128, seed=3).to(dtype)
    x[0, :128] = 0
    x[0, 128:256] = info.max
    x[0, 256] = info.max
    x[0, 384:512] = info.smallest_normal
    x[0, 512:640] = info.smallest_normal * info.eps          # the smallest subnormal
    x[0, 640:768] *= 1e-30 if dtype != torch.float16 else 1e-6
    x[0, 800] = float("inf")
    x[0, 900] = float("-inf")
    x[0, 1100] = float("nan")
    x[0, 1152:1280] = -0.0
    x[0, 1281] = -info.max
    _same_bytes(ecw.fp8_quantize(x.cuda()), _f64(x))
    assert torch.isnan(ecw.fp8_quantize(x.cuda()).dequantize(torch.float32)[0, 768:1152]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantise_strides_and_offsets(dtype):
    big = _randn(9, 700, seed=5).to(dtype).cuda()
    for x in (big[:, 1:334], big[::2, 3:], big[2:3, 5:6], big[:, :130], big[:1].expand(4, 700), big[3, 7:400]):
        _same_bytes(ecw.fp8_quantize(x), _f64(x if x.dim() == 2 else x[None]))
    out = ecw.fp8_quantize(big[:2, :40])
    given = ecw.FP8Tensor(torch.full_like(out.codes, 9), torch.full_like(out.scales, 9), 2, 40)
    assert ecw.fp8_quantize(big[:2, :40], out=given) is given
    assert torch.equal(given.codes, out.codes) and torch.equal(given.scales, out.scales)


def test_dequantise_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (246, 1))
    scales = np.full((246, 16), 127, np.uint8)
    scales[:, 0] = np.arange(10, 256)
    scales[:, 1] = np.arange(10, 256)[::-1]
    t = ecw.FP8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 246, 256)
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(R.values(codes, scales[:, :2], 256))
    for dtype in DTYPES:  # past s = 119 some values pass fp32's range: infinite there
        assert torch.equal(t.dequantize(dtype).cpu().nan_to_num(7.0, 9e9, -9e9), want.to(torch.float32).to(dtype).nan_to_num(7.0, 9e9, -9e9))


# silu and its product in fp32: e^-g and the reciprocal within 2^-23 each, three more
# roundings of 2^-24, so 3.5 * 2^-23 < 2^-21.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 128), (2, 1003), (130, 4096)])
def test_gated(dtype, rows, cols):
    both = (3 * _randn(rows, 2 * cols, seed=cols)).to(dtype)
    both[0, 0] = -80.0
    both[-1, cols - 1] = 80.0
    both = both.cuda()
    gate, x = both[:, :cols], both[:, cols:]
    t = ecw.fp8_quantize(x, gate=gate)
    g = _f64(gate)
    want = _f64(x) * g / (1 + np.exp(-g))
    assert R.between(_f64(t.dequantize(torch.float32)), want, 2.0 ** -21).all()
    assert (t.scales.cpu().numpy()[:, -(-cols // 128):] == 127).all()


def test_gate_of_infinity_and_nan():
    x, g = torch.ones(1, 640, device="cuda"), torch.ones(1, 640, device="cuda")
    g[0, 3], g[0, 130], g[0, 260], x[0, 390] = float("inf"), float("-inf"), float("nan"), float("inf")
    g[0, 513] = -1e4  # a gate that is shut
    v = ecw.fp8_quantize(x, gate=g).dequantize(torch.float32)[0].view(5, 128)
    assert torch.isnan(v[:4]).all() and torch.isfinite(v[4]).all() and v[4, 1] == 0


# ------------------------------------------------------------------ product
def _whole(rows, cols, most, seed, spread=0):
    """Whole numbers up to `most` and a power of two per block: exact in the format."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-most, most + 1, (rows, cols), generator=g).float()
    s = torch.randint(0, spread + 1, (rows, -(-cols // 128)), generator=g).float()
    return v * torch.exp2(s).repeat_interleave(128, 1)[:, :cols]


SHAPES = [(1, 1, 1), (1, 64, 128), (2, 17, 129), (3, 100, 1000), (5, 16, 2048), (16, 33, 2049), (17, 130, 385), (33, 300, 640),
          (40, 4096, 1024), (48, 70, 4100), (64, 65, 257), (65, 257, 300), (100, 513, 2176), (129, 1000, 1023), (200, 64, 8192),
          (257, 384, 1152), (300, 2048, 512), (513, 520, 260), (1003, 1024, 384), (31, 5000, 130), (1, 8192, 4096), (1100, 2305, 128)]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_product_of_whole_numbers_is_exact(batch, rows, cols):
    """Products and sums are whole numbers under 2^24 (3 * 3 * 4 * cols at most), so every
    order of summing them gives the same fp32 number."""
    x, w = _whole(batch, cols, 3, 1, 1), _whole(rows, cols, 3, 2, 1)
    xt, wt = ecw.fp8_quantize(x.cuda()), ecw.fp8_quantize(w.cuda())
    assert torch.equal(xt.dequantize(torch.float32).cpu(), x)
    want = (x.double() @ w.double().t()).float()
    assert want.abs().max() < 2 ** 24
    assert torch.equal(wt.gemm(xt).cpu(), want)
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(wt.gemm(xt, out_dtype=dtype).cpu(), want.to(dtype))


@pytest.mark.parametrize("batch,rows,cols", [(2048, 9000, 256), (4096, 4700, 130), (300, 14336, 512), (1500, 3001, 640), (17, 20000, 257),
                                             (16, 16, 30000), (4, 300, 20000), (40, 100, 25000), (33, 63, 20000), (19, 1, 9000),
                                             (70, 2, 30000), (1, 3, 20001), (130, 130, 16385), (2048, 9000, 4096), (1043, 14511, 1800),
                                             (538, 13235, 2300), (1000, 9000, 4000)])
@pytest.mark.parametrize("out", DTYPES)
def test_large_products_of_whole_numbers_are_exact(batch, rows, cols, out):
    """Tiles of every kind, rounds that are cut, columns in parts; the reference, fp32 sums of
    the same whole numbers under 2^24, is exact on the GPU too."""
    most = 3 if cols < 10000 else 1
    x, w = _whole(batch, cols, most, 1, 1).cuda(), _whole(rows, cols, most, 2, 1).cuda()
    want = x @ w.t()
    assert want.abs().max() < 2 ** 24
    assert torch.equal(ecw.fp8_quantize(w).gemm(ecw.fp8_quantize(x), out_dtype=out), want.to(out))


@pytest.mark.parametrize("batch,rows,cols", [(1, 1024, 4096), (6, 333, 14336), (40, 256, 5000), (130, 200, 2000), (513, 700, 1500)])
@pytest.mark.parametrize("out", DTYPES)
def test_product_of_real_numbers(batch, rows, cols, out):
    """fp32 sums of `cols` exact products, in any order and truncated or rounded: each addition
    is off by at most 2^-23 of the sums' magnitudes; then half a step of the output.  With a
    16-bit output up to 16 products may be added with 12 fraction bits under the largest one's
    power of two: 16 * 2^-12 of it at most is lost."""
    x, w = _randn(batch, cols, seed=4), _randn(rows, cols, seed=5) * torch.exp2(3 * _randn(rows, 1, seed=6))
    x[:, ::50] *= 100
    x[:, 200:300] *= 1e-4
    xt, wt = ecw.fp8_quantize(x.cuda()), ecw.fp8_quantize(w.cuda())
    xv, wv = R.rounded(x.double().numpy()), R.rounded(w.double().numpy())
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    got = _f64(wt.gemm(xt, out_dtype=out))
    tol = (cols * 2.0 ** -23 + (0 if out == torch.float32 else 2.0 ** -8)) * size + torch.finfo(out).eps / 2 * np.abs(want)
    past = np.isinf(got)  # a sum past the output's range (fp16: 65504) is infinite there, of its own sign
    assert (np.abs(want) + tol >= torch.finfo(out).max)[past].all() and (np.sign(got) == np.sign(want))[past].all()
    got, want, size, tol = got[~past], want[~past], size[~past], tol[~past]
    assert (np.abs(got - want) <= tol).all()
    # the error's 2-norm stays at that of rounding errors that do not all point one way
    rounding = torch.finfo(out).eps / 2 if out != torch.float32 else 0
    assert np.linalg.norm(got - want) <= (rounding + 2.0 ** -20) * np.linalg.norm(size)


@pytest.mark.parametrize("batch", [1, 20, 70, 300])
def test_product_with_nan_blocks(batch):
    """A NaN block of w is NaN in its row's outputs, one of x in its own row; no others."""
    x, w = _whole(batch, 300, 3, 1), _whole(40, 300, 3, 2)
    x[batch - 1, 290], w[7, 5], w[39, 130] = float("inf"), float("nan"), float("-inf")
    y = ecw.fp8_quantize(w.cuda()).gemm(ecw.fp8_quantize(x.cuda())).cpu()
    bad = torch.zeros(batch, 40, dtype=torch.bool)
    bad[batch - 1] = True
    bad[:, [7, 39]] = True
    assert torch.equal(torch.isnan(y), bad)
    x[batch - 1, 256:], w[7, :128], w[39, 128:256] = 0, 0, 0
    assert torch.equal(y[~bad], (x.double() @ w.double().t()).float()[~bad])


@pytest.mark.parametrize("batch", [1, 20, 70, 300])
def test_product_with_nan_scales_over_numbers(batch):
    """The scale byte alone makes a block NaN, whatever its codes."""
    x, w = ecw.fp8_quantize(_whole(batch, 300, 3, 1).cuda()), ecw.fp8_quantize(_whole(40, 300, 3, 2).cuda())
    x.scales[0, 2] = 255
    w.scales[11, 0] = 255
    bad = torch.zeros(batch, 40, dtype=torch.bool)
    bad[0], bad[:, 11] = True, True
    assert torch.equal(torch.isnan(w.gemm(x)).cpu(), bad)


@pytest.mark.parametrize("batch", [1, 30, 90])
def test_product_at_the_ends_of_the_range(batch):
    """Scales at both ends of their range: sums that pass fp32 are infinite, products under it vanish."""
    big = ecw.fp8_quantize(torch.full((batch, 256), 3e38, device="cuda"))
    small = ecw.fp8_quantize(torch.full((32, 256), 2.0 ** -100, device="cuda"))
    got = small.gemm(big).cpu()
    v = R.rounded(np.full((1, 256), np.float64(np.float32(3e38))))[0, 0]
    assert torch.equal(got, torch.full((batch, 32), float(np.float32(v * 2.0 ** -100 * 256))))
    assert torch.isinf(ecw.fp8_quantize(torch.full((32, 256), 3e38, device="cuda")).gemm(big)).all()
    assert (small.gemm(ecw.fp8_quantize(torch.full((batch, 256), 2.0 ** -100, device="cuda"))) == 0).all()


def test_product_rows_past_the_end_are_not_written():
    for batch, rows in ((3, 50), (20, 70), (70, 130), (300, 260)):
        x, w = _whole(batch, 200, 2, 1), _whole(rows, 200, 2, 2)
        whole = torch.full((batch + 2, rows), 7.0, device="cuda")
        y = whole[1:-1]
        if y.data_ptr() % 16:
            continue
        ecw.fp8_quantize(w.cuda()).gemm(ecw.fp8_quantize(x.cuda()), y=y)
        assert torch.equal(y.cpu(), (x.double() @ w.double().t()).float())
        assert (whole[0] == 7).all() and (whole[-1] == 7).all()


def test_empty():
    x = torch.zeros(0, 200, device="cuda")
    t = ecw.fp8_quantize(x)
    assert t.shape == (0, 200) and t.dequantize().shape == (0, 200)
    w = ecw.fp8_quantize(torch.ones(8, 200, device="cuda"))
    assert w.gemm(t).shape == (0, 8) and t.gemm(w).shape == (8, 0)


def test_refusals():
    x = torch.ones(4, 256, device="cuda")
    t = ecw.fp8_quantize(x)
    for call, error in [
            (lambda: ecw.fp8_quantize(x.double()), TypeError), (lambda: ecw.fp8_quantize(x.t()), TypeError),
            (lambda: ecw.fp8_quantize(x[None]), ValueError), (lambda: ecw.fp8_quantize(x[:, :0]), ValueError),
            (lambda: ecw.fp8_quantize(x, gate=x[:2]), ValueError), (lambda: ecw.fp8_quantize(x, gate=x.half()), ValueError),
            (lambda: ecw.fp8_quantize(x, gate=x.cpu()), TypeError), (lambda: ecw.fp8_quantize(x, out=x), TypeError),
            (lambda: ecw.fp8_quantize(x[:2], out=t), ValueError), (lambda: t.gemm(x), TypeError),
            (lambda: t.gemm(ecw.fp8_quantize(x[:, :128])), ValueError), (lambda: t.gemm(t, out_dtype=torch.float64), TypeError),
            (lambda: t.gemm(t, y=torch.zeros(4, 5, device="cuda")), ValueError),
            (lambda: t.dequantize(torch.int8), TypeError),
            (lambda: ecw.FP8Tensor(t.codes, t.scales, 4, 257), ValueError),
            (lambda: ecw.FP8Tensor(t.codes[:, ::2], t.scales, 4, 128), TypeError)]:
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("batch", [1, 40, 200])
def test_streams_and_graphs(batch):
    """On another stream, and captured: every replay is the eager result on its inputs."""
    w = ecw.fp8_quantize(_randn(500, 1000, seed=1).cuda())
    x, g = _randn(batch, 1000, seed=2).cuda(), _randn(batch, 1000, seed=3).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = w.gemm(ecw.fp8_quantize(x, gate=g, stream=side), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, w.gemm(ecw.fp8_quantize(x, gate=g)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w.gemm(ecw.fp8_quantize(x, gate=g), out_dtype=torch.bfloat16)
    for seed in (5, 6, 7):
        x.copy_(_randn(batch, 1000, seed=seed))
        want = w.gemm(ecw.fp8_quantize(x, gate=g), out_dtype=torch.bfloat16)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_gate_and_operand_may_be_the_same_tensor():
    x = _randn(5, 300, seed=1).cuda()
    t = ecw.fp8_quantize(x, gate=x)
    assert R.between(_f64(t.dequantize(torch.float32)), _f64(x) ** 2 / (1 + np.exp(-_f64(x))), 2.0 ** -21).all()
    wide = _randn(5, 900, seed=2).cuda()  # a gate whose rows lie otherwise than x's
    t = ecw.fp8_quantize(x, gate=wide[:, 3:303])
    assert torch.equal(t.codes, ecw.fp8_quantize(x, gate=wide[:, 3:303].contiguous()).codes)
    w = _whole(40, 300, 3, 1)
    q = ecw.fp8_quantize(w.cuda())
    assert torch.equal(q.gemm(q).cpu(), (w.double() @ w.double().t()).float())


@pytest.mark.parametrize("batch", [3, 40, 300])
def test_two_streams_and_two_graphs_at_once(batch):
    """Calls that overlap share nothing: the same weights on two streams, and two graphs of them
    replayed in turn."""
    w = ecw.fp8_quantize(_whole(100, 20000, 1, 1).cuda())
    xs = [ecw.fp8_quantize(_whole(batch, 20000, 1, 2 + i).cuda()) for i in range(2)]
    want = [w.gemm(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(w.gemm(xs[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    graphs, held = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            held.append(w.gemm(xs[i]))
    for _ in range(3):
        for y in held:
            y.zero_()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                streams[i].wait_stream(torch.cuda.default_stream())
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(held[i], want[i]) for i in range(2))


def test_offsets_past_32_bits():
    """Rows that lie more than 2^32 bytes behind the first: as by themselves."""
    rows, cols = 66000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:64], x[-64:] = _randn(64, cols, seed=1).cuda(), _randn(64, cols, seed=2).cuda()
    t = ecw.fp8_quantize(x)
    last = ecw.fp8_quantize(x[-64:])
    assert torch.equal(t.codes[-64:], last.codes) and torch.equal(t.scales[-64:], last.scales)
    assert torch.equal(t.dequantize(torch.bfloat16, out=x)[-64:], last.dequantize(torch.bfloat16))
    del x
    for batch in (1, 40, 200):
        a = ecw.fp8_quantize(_randn(batch, cols, seed=3).cuda())
        for out in (torch.float32, torch.bfloat16):
            y, own = t.gemm(a, out_dtype=out)[:, -64:].float(), last.gemm(a, out_dtype=out).float()
            # other tiles, so other orders of the same sums: 2^-12 of the largest, and a step of the output
            assert (y - own).abs().max() <= (2.0 ** -12 + torch.finfo(out).eps) * own.abs().max()


def test_codes_and_scales_are_tensors_of_their_own():
    """They share a piece of memory, and no byte of it; writing into them advances their versions."""
    x = _randn(7, 300, seed=1).cuda()
    t = ecw.fp8_quantize(x)
    assert t.codes.is_contiguous() and t.scales.is_contiguous() and t.scales.data_ptr() % 16 == 0
    assert t.codes.data_ptr() + t.codes.numel() <= t.scales.data_ptr()
    kept, before = t.scales.clone(), (t.codes._version, t.scales._version)
    codes = t.codes.clone()
    t.codes.fill_(3)
    assert torch.equal(t.scales, kept)
    ecw.fp8_quantize(x, out=t)
    assert torch.equal(t.codes, codes) and t.codes._version > before[0] + 1 and t.scales._version > before[1]
    part = ecw.FP8Tensor(t.codes[2:5], t.scales[2:5], 3, 300)
    assert torch.equal(part.dequantize(torch.float32), t.dequantize(torch.float32)[2:5])
    with torch.inference_mode():
        assert ecw.fp8_quantize(x).codes.is_inference() and ecw.rms_norm(x).is_inference()
    keep = t.scales
    del t, part  # the memory lives as long as one of them
    torch.empty(7 * 384, dtype=torch.uint8, device="cuda").fill_(9)
    assert torch.equal(keep, kept)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gate_up_to_where_the_exponential_passes_fp32(dtype):
    """e^-g is a number up to g = -88.72, so the gate is one too, though 1 + e^-g has a reciprocal
    under 2^-126 from -87.34 on; behind -88.73 it is zero.  Blocks of such gates alone."""
    shut = torch.tensor([-87.0, -87.3, -87.33, -87.34, -87.4, -87.5, -87.9, -88.0, -88.1, -88.3, -88.5, -88.6, -88.7]).to(dtype)
    shut = shut[shut > -88.722]  # -88.7 in bf16 is -88.5
    g = shut[torch.arange(3 * 128) % len(shut)].view(3, 128)
    x = ((_randn(3, 128, seed=1).abs() + 0.5) * torch.tensor([[1.0], [-100.0], [1e4 if dtype == torch.float16 else 1e30]])).to(dtype)
    t = ecw.fp8_quantize(x.cuda(), gate=g.cuda())
    want = _f64(x) * _f64(g) / (1 + np.exp(-_f64(g)))
    assert R.between(_f64(t.dequantize(torch.float32)), want, 2.0 ** -21).all()
    g = torch.tensor([-88.75, -89.0, -100.0, -1000.0, -60000.0]).to(dtype)
    t = ecw.fp8_quantize(torch.full((1, 5), 100.0, dtype=dtype, device="cuda"), gate=g[None].cuda())
    assert (t.dequantize(torch.float32) == 0).all()


def test_gate_of_the_largest_and_smallest_numbers():
    """Neither a large nor a small gate leaves fp32's range on the way."""
    g = torch.tensor([[3.4e38, 1e38, 2.0 ** 126, 2.0 ** 125, 1e30] * 26, [2.0 ** -126, -2.0 ** -126, 2.0 ** -120, 1e-30, -1e-30] * 26])[:, :128].contiguous()
    x = torch.tensor([[1.0], [1e35]]).expand(2, 128).contiguous()
    t = ecw.fp8_quantize(x.cuda(), gate=g.cuda())
    want = _f64(x) * _f64(g) / (1 + np.exp(-np.minimum(_f64(g), 700)))
    assert R.between(_f64(t.dequantize(torch.float32)), want, 2.0 ** -21).all()
