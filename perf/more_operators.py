"""Cases of the 8-bit operators and of the rotary positions: quantisation into 8-bit
floats (with a SiLU gate in the same pass), the root-mean-square norm with the residual's
addition and an 8-bit output, the product of two 8-bit matrices, and the rotation of
queries and keys by positions on one axis or several.

The 8-bit format: 128 neighbouring columns of a row form a block with one power-of-two
scale 2^s and 128 E4M3 numbers (three mantissa bits, largest 448).  s is the smallest
whole number with largest magnitude <= 448 * 2^s, held to -117..119 (0 for a block of
zeros); numbers round to nearest, ties to even, and magnitudes over 448 become 448.  A
block that holds an infinity or a NaN stands for NaN.  A last block may be partial.

`own` false: plain torch.  `own` true: this repository's kernels.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def _lib():
    import entropy_coded_weight_amd as ecw
    return ecw


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's gate and up projections on their way into the down projection: latency
        {"name": "quantise-gated-token", "op": "quantise", "rows": 1, "cols": 14336, "dtype": "bf16", "gated": True},
        # the same of a prompt of odd length
        {"name": "quantise-gated-prompt", "op": "quantise", "rows": 2003, "cols": 14336, "dtype": "bf16", "gated": True},
        # a gate/up projection's weights, quantised once when a model is loaded
        {"name": "quantise-weight", "op": "quantise", "rows": 14336, "cols": 4096, "dtype": "bf16", "gated": False},
        # one token's attention output onto the residual stream, and the norm before the feed-forward: latency
        {"name": "norm-token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": "bf16", "out": "fp8"},
        # the same of a long prompt, with the residual stream in 32 bits
        {"name": "norm-prompt", "op": "norm", "rows": 8191, "cols": 4096, "dtype": "bf16", "residual": "fp32",
         "out": "fp8"},
        # the norm of each query head of a prompt, no residual
        {"name": "norm-heads", "op": "norm", "rows": 32096, "cols": 128, "dtype": "fp16", "residual": "none",
         "out": "same"},
        # one decode step of one sequence through a gate/up projection
        {"name": "product-token", "op": "product", "batch": 1, "rows": 14336, "cols": 4096, "out": "bf16"},
        # a decode step of forty sequences through a down projection
        {"name": "product-step", "op": "product", "batch": 40, "rows": 4096, "cols": 14336, "out": "fp32"},
        # a prompt of odd length through a square projection
        {"name": "product-prompt", "op": "product", "batch": 1003, "rows": 4096, "cols": 4096, "out": "bf16"},
        # a long prompt through a gate/up projection
        {"name": "product-long", "op": "product", "batch": 4096, "rows": 14336, "cols": 4096, "out": "bf16"},
        # a decode step of eight sequences far into their contexts: latency
        {"name": "rotary-token", "op": "rotary", "rows": 8, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 128, "axes": 1, "neighbours": False, "base": 500000.0, "top": 131072, "dtype": "bf16"},
        # a prompt with pictures and a film: time, height and width
        {"name": "rotary-pictures", "op": "rotary", "rows": 8191, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 128, "axes": 3, "neighbours": False, "base": 1000000.0, "top": 8192, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "product", "product", "rotary"])
    if op == "quantise":
        cols = _spread(rng, 33, 16384)
        return {"op": op, "rows": _spread(rng, 1, min(16384, 28_000_000 // cols)), "cols": cols,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "gated": rng.choice([False, True])}
    if op == "norm":
        cols = _spread(rng, 33, 16384)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        return {"op": op, "rows": _spread(rng, 1, min(32768, 33_000_000 // cols)), "cols": cols, "dtype": dtype,
                "residual": rng.choice(["none", dtype, "fp32"]), "out": rng.choice(["fp8", "fp8", "same"])}
    if op == "product":
        rows, cols = _spread(rng, 64, 16384), _spread(rng, 64, 16384)
        batch = _spread(rng, 1, max(1, min(4096, 240_000_000_000 // (rows * cols))))
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "out": rng.choice(["fp32", "bf16", "fp16"])}
    dim, heads = rng.choice([64, 80, 96, 128, 192, 256]), rng.choice([1, 2, 3, 4, 8])
    q_heads = heads * rng.choice([1, 2, 3, 4, 8])
    return {"op": op, "rows": _spread(rng, 1, min(16384, 41_000_000 // ((q_heads + heads) * dim))), "q_heads": q_heads,
            "kv_heads": heads, "head_dim": dim, "rotary_dim": rng.choice([dim, dim, dim // 2]),
            "axes": rng.choice([1, 2, 3]), "neighbours": rng.choice([False, True]),
            "base": rng.choice([10000.0, 500000.0, 1000000.0]), "top": _spread(rng, 16, 1048576),
            "dtype": rng.choice(["bf16", "fp16", "fp32"])}


def _size(name):
    return 4 if name == "fp32" else 2


def work(case):
    op = case["op"]
    if op == "quantise":  # in, and the values out
        e = case["rows"] * case["cols"]
        return {"bytes": e * _size(case["dtype"]) * (2 if case["gated"] else 1) + 2 * e, "flops": (8 if case["gated"] else 2) * e}
    if op == "norm":
        e = case["rows"] * case["cols"]
        stream = 0 if case["residual"] == "none" else 2 * _size(case["residual"])
        return {"bytes": e * (_size(case["dtype"]) + stream + (2 if case["out"] == "fp8" else _size(case["dtype"]))),
                "flops": 6 * e}
    if op == "product":
        b, n, k = case["batch"], case["rows"], case["cols"]
        return {"bytes": (n + b) * (k + k / 128) + b * n * _size(case["out"]), "flops": 2 * b * n * k}
    e = case["rows"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
    return {"bytes": 2 * e * _size(case["dtype"]) + 4 * case["axes"] * case["rows"], "flops": 3 * e}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols, dtype):
    """Unit normal, with a few columns twenty times as large, as models have them."""
    x = _normal(g, rows, cols)
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _weights(g, rows, cols, dtype):
    return (_normal(g, rows, cols) * (0.02 * torch.exp2(_normal(g, rows, 1)))).to(dtype)


def _quantise_inputs(case, seed):
    """x, and the gate or None: both are halves of one projection's output."""
    g, rows, cols, dtype = _generator(seed), case["rows"], case["cols"], DTYPE[case["dtype"]]
    if not case["gated"]:
        return (_activations if rows < 64 else _weights)(g, rows, cols, dtype), None
    both = (2 * _normal(g, rows, 2 * cols)).to(dtype)
    return both[:, cols:], both[:, :cols]


def _norm_inputs(case, seed):
    """x, the norm's weight, and the residual stream or None."""
    g, rows, cols, dtype = _generator(seed), case["rows"], case["cols"], DTYPE[case["dtype"]]
    x = _normal(g, rows, cols).to(dtype)
    w = (1 + 0.2 * _normal(g, cols)).to(dtype)
    return x, w, None if case["residual"] == "none" else _activations(g, rows, cols, DTYPE[case["residual"]])


def _product_inputs(case, seed):
    g = _generator(seed)
    return _weights(g, case["rows"], case["cols"], torch.bfloat16), _activations(g, case["batch"], case["cols"], torch.bfloat16)


def _inv_freq(case):
    return case["base"] ** (-torch.arange(0, case["rotary_dim"], 2, dtype=torch.float64) / case["rotary_dim"])


def _sections(case):
    """How many frequencies each axis has, one after the other: about a quarter for the first of three."""
    half, axes = case["rotary_dim"] // 2, case["axes"]
    if axes == 1:
        return [half]
    first = half // 4 if axes == 3 else half // 2
    second = (half - first) // 2 if axes == 3 else half - first
    return [first, second, half - first - second][:axes]


def _rotary_inputs(case, seed):
    g, rows = _generator(seed), case["rows"]
    q = _normal(g, rows, case["q_heads"], case["head_dim"]).to(DTYPE[case["dtype"]])
    k = _normal(g, rows, case["kv_heads"], case["head_dim"]).to(DTYPE[case["dtype"]])
    return q, k, torch.randint(0, case["top"], (case["axes"], rows), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "quantise":
        s["x"], s["gate"] = _quantise_inputs(case, seed)
    elif case["op"] == "norm":
        s["x"], s["weight"], s["residual"] = _norm_inputs(case, seed)
    elif case["op"] == "product":  # w in 8 bits from when the model was loaded, x from the norm before
        w, x = _product_inputs(case, seed)
        s["w"], s["x"] = (_lib().fp8_quantize(t) if own else _quantise(t) for t in (w, x))
    else:
        s["q"], s["k"], s["positions"] = _rotary_inputs(case, seed)
        if own:
            s["rotary"] = _lib().Rotary(case["head_dim"], rotary_dim=case["rotary_dim"], base=case["base"],
                                        sections=_sections(case), neighbours=case["neighbours"])
        else:
            s["inv_freq"] = _inv_freq(case).cuda()
            s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_sections(case))).cuda()
    return s


# ------------------------------------------------------------------ plain forms
def _power(s):
    """2^s as float32, exactly, for whole s in -126..127 (a library's exp2 may round)."""
    return ((s.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 numbers [rows, blocks, 128], scales 2^s [rows, blocks, 1] of x, and its columns."""
    cols = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -cols % 128)).unflatten(-1, (-1, 128))
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    s = torch.where(top > 0, e - torch.where(m > 0.875, 8, 9), 0).clamp(-117, 119)
    bad = ~torch.isfinite(top)
    s = torch.where(bad, 0, s)
    return (x * _power(-s)).clamp(-448, 448).to(torch.float8_e4m3fn), torch.where(bad, math.nan, _power(s)), cols


def _values(codes, scales, cols):
    return (codes.float() * scales).flatten(-2)[..., :cols]


def _rotate(x, cos, sin, c):
    """x [rows, heads, head_dim] by cos and sin [rows, 1, pairs], in 32 bits."""
    half, wide = c["rotary_dim"] // 2, c["rotary_dim"]
    x = x.float()
    a, b = (x[..., :wide:2], x[..., 1:wide:2]) if c["neighbours"] else (x[..., :half], x[..., half:wide])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["neighbours"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., wide:]], -1)


def run(s):
    c = s["case"]
    if c["op"] == "quantise":
        if own:
            return _lib().fp8_quantize(s["x"], gate=s["gate"]).dequantize(torch.bfloat16)
        x = s["x"].float()
        if c["gated"]:
            g = s["gate"].float()
            x = g / (1 + torch.exp(-g)) * x
        return _values(*_quantise(x)).to(torch.bfloat16)
    if c["op"] == "norm":
        if own:
            got = _lib().rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                  out_dtype=torch.float8_e4m3fn if c["out"] == "fp8" else None)
            y, h = got if s["residual"] is not None else (got, None)
            y = y.dequantize(torch.bfloat16) if c["out"] == "fp8" else y
            return y if h is None else (y, h)
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        y = _values(*_quantise(y)).to(torch.bfloat16) if c["out"] == "fp8" else y.to(s["x"].dtype)
        return y if s["residual"] is None else (y, h.to(s["residual"].dtype))
    if c["op"] == "product":
        if own:
            return s["w"].gemm(s["x"], out_dtype=DTYPE[c["out"]])
        return torch.mm(_values(*s["x"]), _values(*s["w"]).t()).to(DTYPE[c["out"]])
    if own:
        return s["rotary"](s["q"], s["k"], s["positions"])
    angle = s["positions"].double().t()[:, s["axis"]] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return tuple(_rotate(x, cos, sin, c).to(x.dtype) for x in (s["q"], s["k"]))


# ------------------------------------------------------------------ the definition, in 64 bits
def _two_to(e):
    """2^e in float64, exactly (a library's ldexp may round)."""
    return ((e + 1023) << 52).view(torch.float64)


def _rounded(x):
    """The values that x (last dimension in blocks of 128) stands for in 8 bits, in float64."""
    cols = x.shape[-1]
    whole = torch.zeros(*x.shape[:-1], -(-cols // 128) * 128, dtype=torch.float64, device=x.device)
    whole[..., :cols] = x
    whole = whole.view(*x.shape[:-1], -1, 128)
    top = whole.abs().max(-1, keepdim=True).values
    s = ((top.view(torch.int64) >> 52) - 1023 - 8).clamp(-117, 119)  # of the largest's own power of two
    s = torch.where(top > 448 * _two_to(s), s + 1, s)
    scale = _two_to(torch.where(top == 0, 0, s).clamp(max=119))
    unit = whole / scale
    # steps: an eighth of the number's own power of two, from 2^-6 down always 2^-9
    step = _two_to(((unit.abs().view(torch.int64) >> 52) - 1023).clamp(-6, 9) - 3)
    near = (torch.round(unit / step) * step).clamp(-448, 448) * scale
    near = torch.where(torch.isfinite(top), near, math.nan)
    return near.reshape(*x.shape[:-1], -1)[..., :cols]


def exact(case, seed):
    if case["op"] == "quantise":
        x, gate = _quantise_inputs(case, seed)
        return _rounded(x.double() if gate is None else x.double() * gate.double() * torch.sigmoid(gate.double()))
    if case["op"] == "norm":
        x, w, residual = _norm_inputs(case, seed)
        h = x.double() if residual is None else x.double() + residual.double()
        y = w.double() * h / torch.sqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / case["cols"] + EPS)
        y = _rounded(y) if case["out"] == "fp8" else y
        return y if residual is None else (y, h)
    if case["op"] == "product":
        w, x = _product_inputs(case, seed)
        return _rounded(x.double()) @ _rounded(w.double()).t()
    q, k, positions = _rotary_inputs(case, seed)
    sections, half, out = _sections(case), case["rotary_dim"] // 2, []
    turn = torch.cat([positions[i].double()[:, None] * f.cuda()
                      for i, f in enumerate(torch.split(_inv_freq(case), sections))], -1)
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    for x in (q, k):
        y = x.double().clone()
        first = slice(0, 2 * half, 2) if case["neighbours"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["neighbours"] else slice(half, 2 * half)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)
