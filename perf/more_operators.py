"""Cases of the norms with quantised outputs, the quantiser and the product of
microscaled operands.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes what a program has
in hand before the call, ``run()`` makes one pass: in plain torch operations,
or, where ``own`` is true, through this package. ``exact()`` computes the same
outputs in 64 bits.

Four operators: ``norm`` (bias and residual addition, LayerNorm or RMSNorm, the
result in 8 bits with scales), ``quantize`` (a matrix or its transpose to 8 or
4 bits with scales; what is 4 bits wide is read back as values), ``product``
(two microscaled matrices, rows by rows) and ``linear`` (a norm into a
microscaled format, the product with a projection's weights, the residual added
and the next LayerNorm from the statistics that the product leaves).

Formats, by name: ``fp8_row`` (E4M3, a 32-bit scale a row), ``fp8_block`` (E4M3,
a 32-bit scale for 128 columns), ``mxfp8`` (E4M3, a power of two for 32 columns),
``mxfp4`` (E2M1, the same) and ``nvfp4`` (E2M1, an E4M3 scale for 16 columns,
values multiplied by one factor for the matrix before).
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = {"fp8_block": 128, "mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
FOUR = ("mxfp4", "nvfp4")
TILED = ("mxfp8", "mxfp4", "nvfp4")


# ---- cases ------------------------------------------------------------------

def _norm(name, dtype, rows, hidden, fmt, mode, bias=False, residual=True, eps=1e-5):
    return {"name": name, "op": "norm", "dtype": dtype, "rows": rows, "hidden": hidden, "fmt": fmt,
            "mode": mode, "bias": bias, "residual": residual, "eps": eps}


def _quantize(name, dtype, rows, cols, fmt, transpose=False, wide=0):
    """rows x cols of the result; wide: columns of the tensor that the input is
    a slice of beyond its own."""
    return {"name": name, "op": "quantize", "dtype": dtype, "rows": rows, "cols": cols, "fmt": fmt,
            "transpose": transpose, "wide": wide}


def _product(name, dtype, m, n, k, fmt, bias=False, residual=False):
    return {"name": name, "op": "product", "dtype": dtype, "m": m, "n": n, "k": k, "fmt": fmt,
            "bias": bias, "residual": residual}


def _linear(name, dtype, m, n, k, fmt, mode, eps=1e-5):
    return {"name": name, "op": "linear", "dtype": dtype, "m": m, "n": n, "k": k, "fmt": fmt,
            "mode": mode, "eps": eps}


def listed():
    return [
        # serving: one token of each of 64 sequences, a scale a token
        _norm("norm_fp8row_bf16_64x8192", "bf16", 64, 8192, "fp8_row", "rmsnorm"),
        # a prompt, or a training batch, of the same model
        _norm("norm_fp8row_bf16_16384x8192", "bf16", 16384, 8192, "fp8_row", "rmsnorm"),
        # a UNet's transformer block: LayerNorm with a bias, 10 blocks of 32
        _norm("norm_mxfp8_f16_8192x320", "f16", 8192, 320, "mxfp8", "layernorm", bias=True),
        # odd rows and a last block of 104 columns, 32-bit activations
        _norm("norm_fp8block_f32_4099x1000", "f32", 4099, 1000, "fp8_block", "layernorm",
              residual=False),
        # a training step's gradient, contracted over the tokens in the weights' gradient
        _quantize("quantize_mxfp8_bf16_8192x8192_t", "bf16", 8192, 8192, "mxfp8", transpose=True),
        # weights, once loaded or updated
        _quantize("quantize_nvfp4_f32_1280x8192", "f32", 1280, 8192, "nvfp4"),
        # odd sizes, a slice of a wider tensor
        _quantize("quantize_mxfp4_bf16_2867x1165", "bf16", 2867, 1165, "mxfp4", wide=3),
        # serving: 16 tokens against a projection's weights, where the weights' bytes count
        _product("product_nvfp4_16x8192x8192", "bf16", 16, 8192, 8192, "nvfp4"),
        # a prompt against the same: the largest case
        _product("product_nvfp4_16384x8192x8192", "bf16", 16384, 8192, 8192, "nvfp4"),
        # odd rows and columns in 8 bits, with a bias and a residual
        _product("product_mxfp8_4099x1165x1280", "f16", 4099, 1165, 1280, "mxfp8", bias=True,
                 residual=True),
        # serving, the whole run: norm, projection, residual, next norm
        _linear("linear_nvfp4_bf16_64x8192x8192", "bf16", 64, 8192, 8192, "nvfp4", "rmsnorm"),
        # a training batch of it, wide to narrow
        _linear("linear_mxfp4_bf16_8192x1280x5120", "bf16", 8192, 1280, 5120, "mxfp4", "layernorm"),
    ]


MOST_BYTES = 7 * 16384 * 8192      # what the largest listed norm moves
MOST_FLOPS = 2 * 16384 * 8192 * 8192


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _some(rng, lo, hi):
    """A size: any, or a multiple of 128 or 16, as most models' are."""
    n = _log(rng, lo, hi)
    step = rng.choice([1, 1, 16, 128])
    return max(lo, min(hi, -(-n // step) * step))


def draw(rng):
    op = rng.choice(["norm", "quantize", "product", "linear"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        hidden = _some(rng, 16, 8192)
        residual = rng.random() < 0.7
        rows = max(1, min(_log(rng, 1, 65536), MOST_BYTES // ((4 * SIZE[dtype]) * hidden)))
        case = _norm("", dtype, rows, hidden, rng.choice(["fp8_row", "fp8_block", "mxfp8"]),
                     rng.choice(["layernorm", "rmsnorm"]), bias=rng.random() < 0.3, residual=residual)
    elif op == "quantize":
        cols = _some(rng, 1, 16384)
        rows = max(1, min(_some(rng, 1, 16384), MOST_BYTES // ((4 + 2 * SIZE[dtype]) * cols)))
        case = _quantize("", dtype, rows, cols,
                         rng.choice(["fp8_row", "fp8_block", "mxfp8", "mxfp4", "nvfp4"]),
                         transpose=rng.random() < 0.5, wide=rng.choice([0, 0, 3, 16]))
    else:
        dtype = rng.choice(["bf16", "f16"])
        n, k = _some(rng, 16, 8192), _some(rng, 16, 8192)
        if op == "product":
            m = max(1, min(_log(rng, 1, 32768), MOST_FLOPS // (4 * n * k)))
            case = _product("", dtype, m, n, k, rng.choice(["mxfp8", "mxfp4", "nvfp4"]),
                            bias=rng.random() < 0.4, residual=rng.random() < 0.4)
        else:
            m = max(1, min(_log(rng, 1, 16384), MOST_FLOPS // (8 * n * k)))
            case = _linear("", dtype, m, n, k, rng.choice(["mxfp8", "mxfp4", "nvfp4"]),
                           rng.choice(["layernorm", "rmsnorm"]))
    del case["name"]
    return case


# ---- the formats in plain torch operations ----------------------------------

# E2M1's values in the order of their codes, the sign in the fourth bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
# codes of E2M1 are told apart at these; a value at one goes to the even code
E2M1_STEPS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _padded(cols, fmt):
    """Columns that a row of codes has room for."""
    return -(-cols // 32) * 32 if fmt in TILED else cols


def _blocks(v, size):
    """[rows, cols] with zeros behind the last column, as [rows, blocks, size]."""
    rows, cols = v.shape
    n = -(-cols // size)
    out = torch.zeros((rows, n * size), device=v.device, dtype=v.dtype)
    out[:, :cols] = v
    return out.view(rows, n, size)


def _tile(scales):
    """Scales [rows, blocks] in tiles of 128 rows by 4 blocks, zeros around."""
    rows, n = scales.shape
    r, c = -(-rows // 128), -(-n // 4)
    out = torch.zeros((r * 128, c * 4), device=scales.device, dtype=scales.dtype)
    out[:rows, :n] = scales
    return out.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(tiles, rows, n):
    r, c = tiles.shape[:2]
    return tiles.permute(0, 3, 2, 1, 4).reshape(r * 128, c * 4)[:rows, :n]


def _e4m3(v):
    """Codes (float8) of 32-bit values, to nearest even, 448 at most."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1(v):
    """Codes 0 to 15 of 32-bit values, to nearest even, 6 at most."""
    a = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for i, step in enumerate(E2M1_STEPS):
        code += (a > step) if i % 2 == 0 else (a >= step)
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _pow2(exponents):
    """2^e of whole numbers from -127 to 127, exactly: torch.ldexp goes through a power."""
    e = exponents.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _exponent(amax, most):
    """The least e from -127 on with amax <= most 2^e, for most = 448 or 6."""
    fraction, e = torch.frexp(amax)                  # amax = fraction 2^e, 1/2 <= fraction < 1
    top, k = math.frexp(most)
    return torch.where(amax > 0, (e - k + (fraction > top)).clamp(min=-127), -127)


def _plain_quantize(v, fmt, mul=None):
    """(codes, scales) of 32-bit values [rows, cols]."""
    rows, cols = v.shape
    if fmt in ("fp8_row", "fp8_block"):
        b = v.view(rows, 1, cols) if fmt == "fp8_row" else _blocks(v, 128)
        amax = b.abs().amax(dim=2).clamp(min=2.0 ** -100)
        codes = _e4m3(b * (448.0 / amax)[..., None]).view(rows, -1)[:, :cols].contiguous()
        scales = amax / 448.0
        return codes, scales[:, 0].contiguous() if fmt == "fp8_row" else scales
    size = BLOCK[fmt]
    wide = _padded(cols, fmt)
    if mul is not None:
        v = v * mul
    b = _blocks(v, size)
    amax = b.abs().amax(dim=2)
    if fmt == "nvfp4":
        scales = _e4m3(amax / 6.0)
        s = scales.float()[..., None]
        b = torch.where(s > 0, b / s, torch.zeros_like(b))
        scales = scales.view(torch.uint8)
    else:
        e = _exponent(amax, 448.0 if fmt == "mxfp8" else 6.0)
        b = b * _pow2(-e)[..., None]
        scales = (e + 127).to(torch.uint8)
    tiles = _tile(scales).view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu)
    if fmt == "mxfp8":
        return _e4m3(b).view(rows, -1), tiles
    code = torch.zeros((rows, wide), dtype=torch.uint8, device=v.device)
    code[:, :b.shape[1] * size] = _e2m1(b).view(rows, -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), tiles


def _e8m0(scales):
    return _pow2(scales.view(torch.uint8).to(torch.int32) - 127)


def _plain_values(codes, scales, fmt, rows, cols, mul=None):
    """The 32-bit values [rows, cols] that microscaled codes stand for."""
    size = BLOCK[fmt]
    n = -(-cols // size)
    if fmt == "mxfp8":
        v = codes.float()
    else:
        table = torch.tensor(E2M1, device=codes.device)
        v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=-1).flatten(1)
    s = _untile(scales.view(torch.uint8), rows, n).contiguous()
    s = s.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _e8m0(s)
    v = (v[:, :cols] * s.repeat_interleave(size, dim=1)[:, :cols])
    return v if mul is None else v / mul


# ---- inputs -----------------------------------------------------------------

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).add_(mean).to(DTYPES[dtype])


def _activations(gen, rows, cols, dtype, mean=0.1):
    """Activations as they come out of a block: a few columns are ten times the others."""
    t = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.01
    return t.mul_(torch.where(loud, 10.0, 1.0)).add_(mean).to(DTYPES[dtype])


def _operand(gen, rows, cols, fmt, std):
    """(codes, scales, mul) of normal values, in the public layout."""
    v = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32).mul_(std)
    mul = (2688.0 / v.abs().amax()).reshape(1) if fmt == "nvfp4" else None
    return (*_plain_quantize(v, fmt, mul), mul)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = case["dtype"], case["op"]
    s = {"case": case}
    if op == "norm":
        rows, hidden = case["rows"], case["hidden"]
        s["x"] = _activations(gen, rows, hidden, dt)
        s["residual"] = _activations(gen, rows, hidden, dt) if case["residual"] else None
        s["bias"] = _normal(gen, (hidden,), dt, 0.1) if case["bias"] else None
        s["gamma"] = _normal(gen, (hidden,), dt, 0.05, 1.0)
        s["beta"] = _normal(gen, (hidden,), dt, 0.05) if case["mode"] == "layernorm" else None
    elif op == "quantize":
        shape = (case["rows"], case["cols"])
        if case["transpose"]:
            shape = shape[::-1]
        s["x"] = _activations(gen, shape[0], shape[1] + case["wide"], dt)[:, :shape[1]]
        s["mul"] = (2688.0 / s["x"].abs().amax().float()).reshape(1) if case["fmt"] == "nvfp4" else None
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _operand(gen, m, k, case["fmt"], 1.0)
        s["b"] = _operand(gen, n, k, case["fmt"], k ** -0.5)
        s["bias"] = _normal(gen, (n,), dt, 0.1) if case["bias"] else None
        s["residual"] = _normal(gen, (m, n), dt) if case["residual"] else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["x"], s["residual"] = _activations(gen, m, k, dt), _normal(gen, (m, k), dt)
        s["gamma"] = _normal(gen, (k,), dt, 0.05, 1.0)
        s["beta"] = _normal(gen, (k,), dt, 0.05) if case["mode"] == "layernorm" else None
        s["w"] = _operand(gen, n, k, case["fmt"], k ** -0.5)
        # the factor of a step before: 448 * 6 over the largest |y| that was seen
        s["mul"] = torch.full((1,), 2688.0 / 24.0, device="cuda") if case["fmt"] == "nvfp4" else None
        s["skip"] = _normal(gen, (m, n), dt)
        s["next_gamma"], s["next_beta"] = _normal(gen, (n,), dt, 0.05, 1.0), _normal(gen, (n,), dt, 0.05)
    return s


# ---- the plain forms --------------------------------------------------------

def _plain_norm(x, bias, residual, gamma, beta, mode, eps):
    """(stored sum or None, y in 32 bits, mean or None, rstd)"""
    v, total = x.float(), None
    if bias is not None:
        v = v + bias.float()
    if residual is not None:
        v = v + residual.float()
    if bias is not None or residual is not None:
        total = v.to(x.dtype)
        v = total.float()
    mean = v.mean(dim=1, keepdim=True) if mode == "layernorm" else None
    d = v - mean if mean is not None else v
    rstd = 1 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + eps)
    y = d * rstd * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return total, y, None if mean is None else mean[:, 0], rstd[:, 0]


def _plain_product(a, b, fmt, m, n, k, bias, residual, dtype):
    left = _plain_values(*a[:2], fmt, m, k)
    right = _plain_values(*b[:2], fmt, n, k)
    out = left @ right.T
    if a[2] is not None:
        out = out / (a[2] * b[2])
    if bias is not None:
        out = out + bias.float()
    if residual is not None:
        out = out + residual.float()
    return out.to(dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        total, y, mean, rstd = _plain_norm(s["x"], s["bias"], s["residual"], s["gamma"], s["beta"],
                                           c["mode"], c["eps"])
        codes, scales = _plain_quantize(y, c["fmt"])
        return {"sum": total, "codes": codes, "scales": scales, "mean": mean, "rstd": rstd}
    if c["op"] == "quantize":
        v = (s["x"].T if c["transpose"] else s["x"]).float().contiguous()
        codes, scales = _plain_quantize(v, c["fmt"], s["mul"])
        if c["fmt"] not in FOUR:
            return {"codes": codes, "scales": scales}
        v = _plain_values(codes, scales, c["fmt"], c["rows"], c["cols"], s["mul"])
        return {"values": v.to(torch.bfloat16), "scales": scales}
    m, n, k, dt = c["m"], c["n"], c["k"], DTYPES[c["dtype"]]
    if c["op"] == "product":
        return {"out": _plain_product(s["a"], s["b"], c["fmt"], m, n, k, s["bias"], s["residual"], dt)}
    total, y, _, _ = _plain_norm(s["x"], None, s["residual"], s["gamma"], s["beta"], c["mode"], c["eps"])
    a = (*_plain_quantize(y, c["fmt"], s["mul"]), s["mul"])
    out = _plain_product(a, s["w"], c["fmt"], m, n, k, None, s["skip"], dt)
    _, y, _, _ = _plain_norm(out, None, None, s["next_gamma"], s["next_beta"], "layernorm", c["eps"])
    return {"sum": total, "out": out, "y": y.to(dt)}


# ---- through the package ----------------------------------------------------

def _own(s):
    import normalization_fwd_gb300 as nf
    c = s["case"]
    fmt = c["fmt"]
    if c["op"] == "norm":
        r = nf.fused_norm_quant_fwd(s["x"], s["gamma"], s["beta"], format=fmt, bias=s["bias"],
                                    residual=s["residual"], eps=c["eps"], mode=c["mode"])
        q = r["q"]
        return {"sum": r["sum"], "codes": q.codes, "scales": q.scales, "mean": r["mean"],
                "rstd": r["rstd"]}
    if c["op"] == "quantize":
        q = nf.quantize(s["x"], fmt, mul=s["mul"], transpose=c["transpose"])
        if fmt not in FOUR:
            return {"codes": q.codes, "scales": q.scales}
        return {"values": nf.dequantize(q, torch.bfloat16), "scales": q.scales}
    m, n, k, dt = c["m"], c["n"], c["k"], DTYPES[c["dtype"]]
    if c["op"] == "product":
        a, b = (nf.Quantized(t[0], t[1], fmt, rows, k, t[2]) for t, rows in ((s["a"], m), (s["b"], n)))
        return {"out": nf.scaled_product(a, b, dtype=dt, bias=s["bias"], residual=s["residual"])["out"]}
    r = nf.fused_norm_quant_fwd(s["x"], s["gamma"], s["beta"], format=fmt, mul=s["mul"],
                                residual=s["residual"], eps=c["eps"], mode=c["mode"])
    w = nf.Quantized(s["w"][0], s["w"][1], fmt, n, k, s["w"][2])
    p = nf.scaled_product(r["q"], w, dtype=dt, residual=s["skip"], partials=True)
    y = nf.fused_norm_fwd_from_partials(p["out"], p["psum"], p["psq"], p["tile_cols"],
                                        s["next_gamma"], s["next_beta"], kind="sum_m2",
                                        eps=c["eps"])["y"]
    return {"sum": r["sum"], "out": p["out"], "y": y}


def run(state):
    return _own(state) if own else _plain(state)


def _stored(rows, cols, fmt):
    """Bytes of a matrix's codes and scales."""
    if fmt == "fp8_row":
        return rows * cols + 4 * rows
    if fmt == "fp8_block":
        return rows * cols + 4 * rows * -(-cols // 128)
    return rows * cols // (2 if fmt in FOUR else 1) + rows * -(-cols // BLOCK[fmt])


def work(case):
    es, op, fmt = SIZE[case["dtype"]], case["op"], case["fmt"]
    if op == "norm":
        rows, hidden = case["rows"], case["hidden"]
        n = rows * hidden
        passes = 1 + case["residual"] + (case["residual"] or case["bias"])
        return {"bytes": passes * n * es + _stored(rows, hidden, fmt) + 4 * rows + 3 * hidden * es,
                "flops": 10 * n}
    if op == "quantize":
        n, q = case["rows"] * case["cols"], _stored(case["rows"], case["cols"], fmt)
        return {"bytes": n * es + q + (q + 2 * n if fmt in FOUR else 0), "flops": 4 * n}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "product":
        return {"bytes": _stored(m, k, fmt) + _stored(n, k, fmt) + m * n * es * (1 + case["residual"]),
                "flops": 2 * m * n * k}
    return {"bytes": 3 * m * k * es + 2 * _stored(m, k, fmt) + _stored(n, k, fmt) + 4 * m * n * es,
            "flops": 2 * m * n * k}


# ---- 64 bits ----------------------------------------------------------------

def _two(e):
    """2^e in 64 bits, for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_grid(v, bits, least, most):
    """The nearest value with `bits` bits behind the leading one and steps of
    2^least at least, ties to even, `most` at most."""
    _, e = torch.frexp(v)
    unit = _two(torch.clamp(e - 1 - bits, min=least))
    return (torch.round(v / unit) * unit).clamp(-most, most)


def _grid_e4m3(v):
    return _to_grid(v, 3, -9, 448.0)


def _grid_e2m1(v):
    return _to_grid(v, 1, -1, 6.0)


def _cut(v, size):
    rows, cols = v.shape
    return torch.nn.functional.pad(v, (0, -cols % size)).reshape(rows, -1, size)


def _exact_quantize(v, fmt, mul=None):
    """(code values [rows, columns with room], scales as the call lays them out,
    values [rows, cols])"""
    rows, cols = v.shape
    if mul is not None:
        v = v * mul.double()
    b = _cut(v, cols if fmt == "fp8_row" else BLOCK[fmt])
    amax = b.abs().amax(dim=2, keepdim=True)
    if fmt in ("fp8_row", "fp8_block"):
        amax = amax.clamp(min=2.0 ** -100)
        s = amax / 448
        # the factor is a 32-bit number
        codes = _grid_e4m3(b * (448 / amax).float().double())
    elif fmt == "nvfp4":
        s = _grid_e4m3(amax / 6)
        codes = _grid_e2m1(b / torch.where(s > 0, s, torch.inf))
    else:
        most = 448.0 if fmt == "mxfp8" else 6.0
        e = torch.ceil(torch.log2(amax / most).clamp(min=-127))
        e = torch.where(most * _two(e - 1) >= amax, e - 1, e).clamp(min=-127)
        s = _two(e)
        codes = (_grid_e4m3 if fmt == "mxfp8" else _grid_e2m1)(b / s)
    values = (codes * s).reshape(rows, -1)[:, :cols]
    if mul is not None:
        values = values / mul.double()
    codes = codes.reshape(rows, -1)
    s = s[..., 0]
    if fmt in TILED:
        codes = codes[:, :_padded(cols, fmt)]
        pad = (0, -s.shape[1] % 4, 0, -rows % 128)
        # what surrounds the scales is a code of 0
        s = torch.nn.functional.pad(s, pad, value=0.0 if fmt == "nvfp4" else 2.0 ** -127)
        s = s.unflatten(0, (-1, 4, 32)).unflatten(3, (-1, 4)).permute(0, 3, 2, 1, 4)
    else:
        codes = codes[:, :cols]
        s = s[:, 0] if fmt == "fp8_row" else s
    return codes, s, values


def _exact_norm(x, bias, residual, gamma, beta, mode, eps):
    v, total = x.double(), None
    if bias is not None or residual is not None:
        # the sum is stored, and what is stored is normalised
        v = x.float() if bias is None else x.float() + bias.float()
        v = v if residual is None else v + residual.float()
        total = v.to(x.dtype).double()
        v = total
    mean = None
    if mode == "layernorm":
        mean = v.sum(dim=1) / v.shape[1]
        v = v - mean[:, None]
    rstd = (v.square().sum(dim=1) / v.shape[1] + eps).pow(-0.5)
    y = torch.einsum("rh,r,h->rh", v, rstd, gamma.double())
    return total, y if beta is None else y + beta.double(), mean, rstd


def _exact_values(codes, scales, mul, fmt, rows, cols):
    size = BLOCK[fmt]
    if fmt == "mxfp8":
        v = codes.double()
    else:
        pair = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(rows, -1).int()
        e, f = (pair >> 1) & 3, pair & 1
        v = torch.where(e > 0, (1.0 + 0.5 * f.double()) * _two(e - 1), 0.5 * f.double())
        v = torch.where(pair >= 8, -v, v)
    s = scales.double() if fmt == "nvfp4" else _two(scales.view(torch.uint8).int() - 127)
    s = s.permute(0, 3, 2, 1, 4).flatten(3, 4).flatten(0, 2)[:rows, :-(-cols // size)]
    v = _cut(v[:, :cols], size) * s[..., None]
    v = v.reshape(rows, -1)[:, :cols]
    return v if mul is None else v / mul.double()


def exact(case, seed):
    s = prepare(case, seed)
    c, fmt = case, case["fmt"]
    if c["op"] == "norm":
        total, y, mean, rstd = _exact_norm(s["x"], s["bias"], s["residual"], s["gamma"], s["beta"],
                                           c["mode"], c["eps"])
        codes, scales, _ = _exact_quantize(y, fmt)
        return {"sum": total, "codes": codes, "scales": scales, "mean": mean, "rstd": rstd}
    if c["op"] == "quantize":
        v = s["x"].double()
        codes, scales, values = _exact_quantize(v.T if c["transpose"] else v, fmt, s["mul"])
        return {"values": values, "scales": scales} if fmt in FOUR else {"codes": codes, "scales": scales}
    m, n, k = c["m"], c["n"], c["k"]
    if c["op"] == "product":
        out = _exact_values(*s["a"], fmt, m, k) @ _exact_values(*s["b"], fmt, n, k).T
        if s["bias"] is not None:
            out += s["bias"].double()
        return {"out": out if s["residual"] is None else out + s["residual"].double()}
    total, y, _, _ = _exact_norm(s["x"], None, s["residual"], s["gamma"], s["beta"], c["mode"], c["eps"])
    out = _exact_quantize(y, fmt, s["mul"])[2] @ _exact_values(*s["w"], fmt, n, k).T + s["skip"].double()
    # the next norm reads the stored row
    stored = out.to(DTYPES[c["dtype"]])
    _, y, _, _ = _exact_norm(stored, None, None, s["next_gamma"], s["next_beta"], "layernorm", c["eps"])
    return {"sum": total, "out": out, "y": y}
