"""Outputs that the caller gives to the 8-bit calls, the norm and the rotary positions: next to what
is read or over it, and what lies around them."""
import pytest
import torch

import entropy_coded_weight_amd as ecw

pytestmark = pytest.mark.gpu
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


DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def _eight(store, at, rows, cols):
    """An FP8Tensor in `store`'s bytes from `at` on: codes, then scales."""
    codes, scales = rows * (-(-cols // 128) * 128), rows * (-(-cols // 2048) * 16)
    part = store[at:at + codes + scales]
    return ecw.FP8Tensor(part[:codes].view(rows, -1), part[codes:].view(rows, -1), rows, cols)


def test_norm_refuses_outputs_across_its_inputs():
    buf, x = _randn(9, 900, seed=1), _randn(8, 512, seed=2)
    t = _eight(torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"), 0, 8, 512)
    kept = buf.clone()
    for call in (lambda: ecw.rms_norm(x, residual=buf[:-1, :512], residual_out=buf[1:, :512]),
                 lambda: ecw.rms_norm(x, residual=buf[1:, :512], residual_out=buf[:-1, :512]),
                 lambda: ecw.rms_norm(buf[:8, 8:520], residual=x, residual_out=buf[:8, :512]),
                 lambda: ecw.rms_norm(buf[:8, :512], residual=buf[:8, 388:], residual_out=buf[:8, 300:812]),
                 lambda: ecw.rms_norm(x, buf[3, :512], residual=x, residual_out=buf[:8, 388:]),
                 lambda: ecw.rms_norm(x, buf[3, 100:612], residual=x, residual_out=buf[:8, 388:]),
                 lambda: ecw.rms_norm(x, out=ecw.FP8Tensor(t.codes, t.codes.view(-1)[:128].view(8, 16), 8, 512)),
                 lambda: ecw.rms_norm(t.codes.view(torch.bfloat16), out=_eight(t.codes.view(-1), 0, 8, 256))):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(buf, kept)


def test_norm_takes_outputs_between_its_inputs():
    x, w = _randn(8, 512, seed=2), _randn(388, seed=4)
    buf = _randn(9, 1800, seed=1)
    kept = buf.clone()
    want, h = ecw.rms_norm(x, residual=kept[:8, :512])
    y, got = ecw.rms_norm(x, residual=buf[:8, :512], residual_out=buf[:8, 512:1024])
    assert torch.equal(y, want) and torch.equal(buf[:8, 512:1024], h) and got.data_ptr() == buf[:, 512:].data_ptr()
    assert torch.equal(buf[:, :512], kept[:, :512]) and torch.equal(buf[:, 1024:], kept[:, 1024:]) and torch.equal(buf[8], kept[8])
    # the row before's free columns, a weight between two rows, and every other row
    buf.copy_(kept)
    buf[3, 1100:1488] = w
    want, h = ecw.rms_norm(x[:, :388], w, residual=kept[1:, :388])
    y, _ = ecw.rms_norm(x[:, :388], buf[3, 1100:1488], residual=buf[1:, :388], residual_out=buf[:8, 512:900])
    assert torch.equal(y, want) and torch.equal(buf[:8, 512:900], h)
    buf.copy_(kept)
    want, h = ecw.rms_norm(x[:4], residual=kept[:8:2, :512])
    y, _ = ecw.rms_norm(x[:4], residual=buf[:8:2, :512], residual_out=buf[1:8:2, :512])
    assert torch.equal(y, want) and torch.equal(buf[1:8:2, :512], h) and torch.equal(buf[::2], kept[::2])


@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 64), (33001, 128), (33001, 40), (9003, 500), (5001, 1000), (2500, 2048), (2101, 4096),
                                       (2050, 8192), (600, 30000)])
def test_norm_in_place_of_many_rows(rows, cols):
    """Each row is read by the lanes that write it and no others: the residual over itself, and the
    result over x, are what they are apart."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    for dtype in (torch.bfloat16, torch.float32):
        r = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
        for out in (EIGHT, torch.bfloat16):
            want, h = ecw.rms_norm(x, residual=r, out_dtype=out)
            over, z = r.clone(), x.clone()
            y, got = ecw.rms_norm(z, residual=over, residual_out=over, **({"out_dtype": out} if out is EIGHT else {"out": z}))
            assert got.data_ptr() == over.data_ptr() and torch.equal(over, h)
            assert torch.equal(y.codes, want.codes) and torch.equal(y.scales, want.scales) if out is EIGHT else torch.equal(z, want)


def test_rotary_refuses_outputs_across_its_inputs():
    qkv = _randn(9, 8, 64, seed=1)
    kept, at, r = qkv.clone(), torch.arange(9, dtype=torch.int32, device="cuda"), ecw.Rotary(64)
    store = torch.zeros(4096, device="cuda")
    for call in (lambda: r(qkv[:, 0:4], None, at, out=qkv[:, 1:5]), lambda: r(qkv[:-1, 0:4], None, at[:8], out=qkv[1:, 0:4]),
                 lambda: r(qkv[:, 0:4], qkv[:, 4:6], at, out=(qkv[:, 0:4], qkv[:, 3:5])),
                 lambda: r(qkv[:, 0:4], qkv[:, 4:6], at, out=(qkv[:, 4:8], None)),
                 lambda: r(qkv[:, 0:2], qkv[:, 2:4], at, out=(qkv[:, 4:6], qkv[:, 5:7])),
                 lambda: r(qkv[:, ::2], None, at, out=qkv[:, 0:4]), lambda: r(qkv[:, 0:4], None, at, out=qkv[:, [3, 2, 1, 0]][:, :1].expand(9, 4, 64)),
                 lambda: r(qkv[:, 0:4], None, at, out=torch.as_strided(store, (9, 4, 64), (64, 64, 1))),
                 lambda: r(qkv[:, 0:4], None, at, out=torch.as_strided(store, (9, 4, 64), (200, 60, 1))),
                 lambda: r(qkv[:, 0:1], None, store.view(torch.int32)[300:309], out=torch.as_strided(store, (9, 1, 64), (64, 64, 1)))):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(qkv, kept)


def test_rotary_takes_outputs_between_its_inputs():
    qkv = _randn(9, 8, 128, seed=1)
    kept, at, r = qkv.clone(), torch.arange(9, dtype=torch.int32, device="cuda") * 100, ecw.Rotary(64)
    for q, out in ((lambda t: t[:, 0:4, :64], lambda t: t[:, 4:8, :64]), (lambda t: t[..., :64], lambda t: t[..., 64:]),
                   (lambda t: t[:, ::2, :64], lambda t: t[:, 1::2, :64]), (lambda t: t[:-1, 4:, 64:], lambda t: t[1:, :4, 64:]),
                   (lambda t: t.transpose(0, 1)[:4, :, :64], lambda t: t.transpose(0, 1)[4:, :, :64])):
        qkv.copy_(kept)
        p = at[:q(kept).shape[0]]
        want = r(q(kept), None, p)
        r(q(qkv), None, p, out=out(qkv))
        assert torch.equal(out(qkv), want)
        out(qkv).copy_(out(kept))
        assert torch.equal(qkv, kept)
    wide = ecw.Rotary(128)
    want = wide(kept[:, 0:4], kept[:, 4:6], at)
    qkv.copy_(kept)
    wide(qkv[:, 0:4], qkv[:, 4:6], at, out=(qkv[:, 0:4], qkv[:, 4:6]))
    assert torch.equal(qkv[:, 0:4], want[0]) and torch.equal(qkv[:, 4:6], want[1]) and torch.equal(qkv[:, 6:], kept[:, 6:])


def test_matrices_refuse_outputs_over_their_inputs():
    store = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    x, g = store[:4096].view(torch.bfloat16).view(8, 256), store[8192:12288].view(torch.bfloat16).view(8, 256)
    t = _eight(store, 16384, 8, 256)
    y = store[32768:].view(torch.float32)
    for call in (lambda: ecw.fp8_quantize(x, out=_eight(store, 2048, 8, 256)), lambda: ecw.fp8_quantize(x, out=_eight(store, 0, 8, 256)),
                 lambda: ecw.fp8_quantize(x, gate=g, out=_eight(store, 6144, 8, 256)),
                 lambda: ecw.fp8_quantize(x, out=ecw.FP8Tensor(t.codes, t.codes.view(-1)[128:256].view(8, 16), 8, 256)),
                 lambda: t.dequantize(out=store[16384 + 512:16384 + 512 + 4096].view(torch.float16).view(8, 256)),
                 lambda: t.dequantize(out=store[18432 + 64:18432 + 64 + 4096].view(torch.float16).view(8, 256)),
                 lambda: t.gemm(t, store[16384:16384 + 256].view(torch.float32).view(8, 8)),
                 lambda: t.gemm(_eight(store, 0, 8, 256), store[1024:1280].view(torch.float32).view(8, 8)),
                 lambda: t.gemm(_eight(store, 0, 8, 256), store[2048:2304].view(torch.float32).view(8, 8)),
                 lambda: _eight(store, 0, 8, 256).gemm(t, store[2048:2304].view(torch.float32).view(8, 8))):
        with pytest.raises(ValueError):
            call()
    assert (store == 0).all()
    x.copy_(_randn(8, 256, seed=1)), g.copy_(_randn(8, 256, seed=2))
    want = ecw.fp8_quantize(x.clone(), gate=g.clone())
    assert ecw.fp8_quantize(x, gate=g, out=t) is t and torch.equal(t.codes, want.codes) and torch.equal(t.scales, want.scales)
    got = t.gemm(t, y[:64].view(8, 8))
    assert got.data_ptr() == y.data_ptr() and torch.equal(got, want.gemm(want)) and (y[64:] == 0).all()


def test_rotary_into_one_tensor_on_another_stream():
    q, at, r = _randn(5, 3, 64, seed=1), torch.arange(5, dtype=torch.int32, device="cuda"), ecw.Rotary(64)
    want, side = r(q, None, at), torch.cuda.Stream()
    y, one = torch.zeros_like(q), torch.zeros_like(q[:, :1])
    side.wait_stream(torch.cuda.current_stream())
    got = r(q, None, at, out=y, stream=side)
    both = r(q, q[:, :1], at, out=(None, one), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, want)
    assert torch.equal(both[0], want) and torch.equal(one, want[:, :1])


def test_refusals_are_the_same_on_a_stream():
    x, side = torch.ones(4, 256, device="cuda"), torch.cuda.Stream()
    t = ecw.fp8_quantize(x)
    for stream in (None, side):
        for call, error in [(lambda: ecw.fp8_quantize(x, out=x, stream=stream), TypeError),
                            (lambda: ecw.fp8_quantize(x, out=[t], stream=stream), TypeError),
                            (lambda: ecw.fp8_quantize([1.0], out=t, stream=stream), ValueError),
                            (lambda: ecw.fp8_quantize(x[:2], out=t, stream=stream), ValueError),
                            (lambda: ecw.rms_norm(x, out=x, out_dtype=EIGHT, stream=stream), TypeError),
                            (lambda: t.gemm(x, stream=stream), TypeError), (lambda: t.gemm(t, y=x, stream=stream), ValueError),
                            (lambda: t.gemm(t, stream=stream, short_sums=True), ValueError)]:
            with pytest.raises(error):
                call()


def _between_guards(shape, dtype, offset=64):
    """A tensor that starts 16-byte aligned and ends right before what must stay 7: (it, all)."""
    n = shape[0] * shape[1]
    store = torch.full((offset + n + 4096,), 7, dtype=dtype, device="cuda")
    y = store[offset:offset + n].view(shape)
    assert y.data_ptr() % 16 == 0
    return y, store


def _untouched(y, store):
    first = y.storage_offset()
    return (store[:first] == 7).all() and (store[first + y.numel():] == 7).all()


@pytest.mark.parametrize("out,short", [(t, False) for t in DTYPES] + [(t, True) for t in DTYPES[:2]])
@pytest.mark.parametrize("batch,rows,cols", [
    (1, 1, 300), (3, 50, 200), (5, 13, 2000), (16, 31, 500), (16, 33, 8192), (17, 70, 200), (20, 70, 200), (40, 63, 20000), (33, 1, 9000),
    (41, 3, 30000), (65, 127, 16384), (70, 130, 200), (129, 257, 300), (300, 260, 200), (301, 259, 4000), (1000, 2049, 130),
    (2049, 4999, 130), (4097, 3585, 128)])
def test_product_writes_its_output_only(batch, rows, cols, out, short):
    """The kernel for few rows, tiles of both instructions, parts of the columns and their join, and
    rounds that are cut: with ragged ends, every element and none before or behind."""
    g = torch.Generator().manual_seed(batch)
    x, w = (torch.randint(-1, 2, (n, cols), generator=g).float().cuda() for n in (batch, rows))
    y, store = _between_guards((batch, rows), out)
    got = ecw.fp8_quantize(w).gemm(ecw.fp8_quantize(x), y=y, short_sums=short)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, (x @ w.t()).to(out))  # whole numbers under 2^24
    assert _untouched(y, store)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (5, 129), (2, 1001), (33, 333), (3, 16390)])
def test_quantise_dequantise_and_norm_write_their_outputs_only(rows, cols, dtype):
    x = _randn(rows, cols, seed=1, dtype=dtype)
    want = ecw.fp8_quantize(x)
    codes, all_codes = _between_guards(tuple(want.codes.shape), torch.uint8)
    scales, all_scales = _between_guards(tuple(want.scales.shape), torch.uint8)
    t = ecw.fp8_quantize(x, out=ecw.FP8Tensor(codes, scales, rows, cols))
    assert torch.equal(codes, want.codes) and torch.equal(scales, want.scales)
    assert _untouched(codes, all_codes) and _untouched(scales, all_scales)
    for out in DTYPES:
        for offset in (64, 67):
            store = torch.full((offset + rows * cols + 100,), 7, dtype=out, device="cuda")
            y = store[offset:offset + rows * cols].view(rows, cols)
            t.dequantize(out=y)
            assert torch.equal(y, want.dequantize(out)) and _untouched(y, store)
            y.fill_(7)
            ecw.rms_norm(x, out=y)
            assert torch.equal(y, ecw.rms_norm(x, out_dtype=out)) and _untouched(y, store)
    want = ecw.rms_norm(x, residual=x, out_dtype=EIGHT)[0]
    wide = torch.full((rows + 2, cols + 9), 7, dtype=dtype, device="cuda")
    ecw.rms_norm(x, residual=x, residual_out=wide[1:-1, 4:-5], out=t)
    assert torch.equal(codes, want.codes) and torch.equal(scales, want.scales)
    assert _untouched(codes, all_codes) and _untouched(scales, all_scales)
    assert torch.equal(wide[1:-1, 4:-5], (x.float() + x.float()).to(dtype))
    wide[1:-1, 4:-5] = 7
    assert (wide == 7).all()
