"""Operators around products in microscaled formats, as work to measure.

A microscaled tensor holds its values in 4 bits (e2m1) or 8 (e4m3) with one power of two for each 32 neighbours of a row.

- the root-mean-square norm with the residual's addition: with its gradients (``rms_norm``, ``rms_norm_grad``), and
  with a microscaled output (``rms_norm_mx``);
- quantisation and back (``quantize_mx``, ``dequantize_mx``);
- products of microscaled operands (``mx_matmul``), and of rows that are quantised on the way (``mx_linear``).

``run`` computes a pass in elementary torch operations where ``own`` is false, and makes the package's
calls where it is true. ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32
EPS = 1e-6


def _spt():
    import software_pipelined_tiled_amd as spt

    return spt


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # 16 sequences decoding one token each: a layer's input norm, written in 8 bits for the next product; launch latency
        dict(name="norm decode", op="norm_mx", rows=16, n=4096, residual=True, dtype="bf16"),
        # the same for a prompt of a larger model
        dict(name="norm prompt", op="norm_mx", rows=8191, n=8192, residual=True, dtype="f16"),
        # a training step's norm, forward and backward, weights kept in 32 bits
        dict(name="norm training", op="norm_train", rows=8192, n=4096, residual=True, dtype="bf16", wtype="f32"),
        # a final norm without a residual, an odd row width, in 32 bits
        dict(name="norm training odd", op="norm_train", rows=1003, n=4097, residual=False, dtype="f32", wtype="f32"),
        # a weight brought to 4 bits
        dict(name="quantize weight", op="quantize", rows=8192, n=8192, bits=4, dtype="bf16"),
        # activations brought to 8 bits, a short last block
        dict(name="quantize odd", op="quantize", rows=301, n=8190, bits=8, dtype="f32"),
        # one token against a square 4-bit weight
        dict(name="product one token", op="product", rows=1, n=8192, k=8192, bits=4, wbits=4, out="bf16"),
        # a decoding batch in 8 bits against a wide 4-bit weight
        dict(name="product batch", op="product", rows=16, n=28672, k=8192, bits=8, wbits=4, out="f16"),
        # a short prompt, rows, columns and depth off the tile sizes
        dict(name="product ragged", op="product", rows=301, n=1025, k=8190, bits=8, wbits=8, out="f32"),
        # a long prompt in 4 bits
        dict(name="product prompt", op="product", rows=8192, n=8192, k=8192, bits=4, wbits=4, out="bf16"),
        # a layer of a decoding batch: its rows quantised to 8 bits and multiplied with a 4-bit weight
        dict(name="linear decode", op="linear", rows=32, n=4096, k=4096, bits=8, wbits=4, dtype="bf16"),
        # a layer of a prompt in 8 bits
        dict(name="linear prompt", op="linear", rows=4096, n=8192, k=4096, bits=8, wbits=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Half of the sizes are multiples of 64, the others any."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm_mx", "norm_train", "quantize", "product", "product", "product", "linear"])
    if op in ("norm_mx", "norm_train", "quantize"):
        n = _size(rng, 100, 28672)
        rows = _log(rng, 1, min(32768, (1 << 26) // n))
        dtype = rng.choice(["bf16", "f16", "f32"] if op != "norm_mx" else ["bf16", "f16"])
        if op == "quantize":
            return dict(op=op, rows=rows, n=n, bits=rng.choice([4, 8]), dtype=dtype)
        case = dict(op=op, rows=rows, n=n, residual=rng.random() < 0.7, dtype=dtype)
        if op == "norm_train":
            case["rows"] = max(1, rows // 2)
            case["wtype"] = rng.choice(["f32", dtype])
        return case
    n, k = _size(rng, 100, 28672), _size(rng, 100, 8192)
    rows = _log(rng, 1, min(16384, int(5.0e11) // (n * k)))
    bits, wbits = rng.choice([(8, 8), (4, 4), (8, 4)])
    if op == "linear":
        return dict(op=op, rows=rows, n=n, k=k, bits=bits, wbits=wbits, dtype=rng.choice(["bf16", "f16"]))
    return dict(op=op, rows=rows, n=n, k=k, bits=bits, wbits=wbits, out=rng.choice(["bf16", "f16", "f32"]))


def _held(rows, k, bits):
    """Bytes of a microscaled tensor."""
    return rows * k * bits / 8 + rows * -(-k // BLOCK)


def _size_of(name):
    return 4 if name == "f32" else 2


def work(case):
    op, rows, n = case["op"], case["rows"], case["n"]
    if op == "norm_mx":  # x (and the residual) in, the sum and the quantised rows out, which come back as values
        es = _size_of(case["dtype"])
        one = rows * n * es
        return {"bytes": one * (3 if case["residual"] else 1) + 2 * _held(rows, n, 8) + 2 * rows * n + n * es, "flops": 6 * rows * n}
    if op == "norm_train":  # x, residual -> h, y; dy, h, dh -> dx
        one, ws = rows * n * _size_of(case["dtype"]), n * _size_of(case["wtype"])
        return {"bytes": one * (8 if case["residual"] else 5) + 3 * ws, "flops": 15 * rows * n}
    if op == "quantize":  # x in, the held values out, and back to values
        return {"bytes": rows * n * _size_of(case["dtype"]) + 2 * _held(rows, n, case["bits"]) + 2 * rows * n, "flops": 2 * rows * n}
    k = case["k"]
    weight = _held(n, k, case["wbits"])
    if op == "product":
        return {"bytes": _held(rows, k, case["bits"]) + weight + rows * n * _size_of(case["out"]), "flops": 2 * rows * n * k}
    return {"bytes": rows * k * 2 + weight + rows * n * 2, "flops": 2 * rows * n * k}


# ----------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(rows, k, g, dtype):
    """Rows as a layer sees them: a few columns are much larger than the others."""
    x = torch.randn((rows, k), generator=g, device="cuda")
    large = torch.rand((k,), generator=g, device="cuda") < 0.005
    return x.mul_(torch.where(large, 20.0, 1.0)).to(dtype)


def _codes(x, bits):
    """A plain quantisation of [rows, k] in the standard's layout: codes as bytes (two 4-bit values in one, the first
    in its low half) and the scales' exponents, with a bias of 127."""
    q, e = _plain_parts(x.float(), bits)
    if bits == 8:
        return q.to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    c = torch.bucketize(q.abs(), levels).to(torch.uint8) + torch.signbit(q).to(torch.uint8) * 8
    if c.shape[1] % 2:
        c = torch.cat([c, torch.zeros_like(c[:, :1])], dim=1)
    return c[:, 0::2] | (c[:, 1::2] << 4), e.to(torch.uint8)


def _inputs(case, seed):
    g = _generator(seed)
    op, rows, n = case["op"], case["rows"], case["n"]
    s = {"op": op, "case": case}
    if op in ("norm_mx", "norm_train"):
        dt = DTYPES[case["dtype"]]
        s["x"] = _activations(rows, n, g, dt)
        s["residual"] = _activations(rows, n, g, dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn((n,), generator=g, device="cuda")).to(DTYPES[case.get("wtype", case["dtype"])])
        if op == "norm_train":
            s["dy"] = _normal((rows, n), g, dt)
            s["dh"] = _normal((rows, n), g, dt) if case["residual"] else None
        return s
    if op == "quantize":
        s["x"] = _activations(rows, n, g, DTYPES[case["dtype"]])
        return s
    k = case["k"]
    x = _activations(rows, k, g, DTYPES[case.get("dtype", "bf16")])
    s["weight"] = _codes(_normal((n, k), g, torch.bfloat16, k ** -0.5), case["wbits"])
    if op == "product":
        s["a"] = _codes(x, case["bits"])
    else:
        s["x"] = x
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] in ("product", "linear"):  # a checkpoint's weight (and the rows that an earlier layer left), laid out once
        k = case["k"]
        s["weight"] = _spt().pack_mx(*s["weight"], case["wbits"], k)
        if case["op"] == "product":
            s["a"] = _spt().pack_mx(*s["a"], case["bits"], k)
    return s


# ------------------------------------------------------------------------------------- plain forms

def _power(e):
    """2 to the power of whole numbers, as fp32's bits: exact, which a library's pow need not be."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _blocks(x):
    """[rows, k] as [rows, blocks, 32], the last block filled with zeros."""
    pad = -x.shape[1] % BLOCK
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.reshape(x.shape[0], -1, BLOCK)


def _plain_parts(x, bits):
    """fp32 rows in units of their scales, rounded to the format's values, [rows, k], and the scales' biased exponents,
    [rows, blocks]. Every step but the rounding to the format is exact."""
    b = _blocks(x)
    field = (b.abs().amax(dim=2).view(torch.int32) >> 23) & 255
    e = torch.clamp(field - (2 if bits == 4 else 8), min=0)
    v = b * _power(127 - e)[:, :, None]
    if bits == 4:  # steps of 0.5 below 2, 1 below 4, 2 up to 6
        mag = v.abs()
        step = torch.where(mag < 2.0, 0.5, torch.where(mag < 4.0, 1.0, 2.0))
        q = torch.clamp(torch.round(mag / step) * step, max=6.0)
    else:  # three bits behind the leading one, steps of 2^-9 below 2^-6
        mag = v.abs()
        lead = (torch.clamp(mag, min=2.0 ** -6).view(torch.int32) & 0x7F800000).view(torch.float32)
        step = lead * 0.125
        q = torch.clamp(torch.round(mag / step) * step, max=448.0)
    q = torch.copysign(q, v)
    return q.reshape(x.shape[0], -1)[:, : x.shape[1]], e


def _plain_values(q, e):
    """The fp32 values of rows in units of their scales."""
    b = _blocks(q)
    v = b * _power(e - 126)[:, :, None] * 0.5  # a scale of 2^-127 is no normal number
    return v.reshape(q.shape[0], -1)[:, : q.shape[1]]


def _plain_decode(codes, e, bits, k):
    """fp32 values of codes in the standard's layout."""
    if bits == 8:
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        levels = torch.cat([levels, -levels])
        q = torch.stack([levels[(codes & 15).int()], levels[(codes >> 4).int()]], dim=2).reshape(codes.shape[0], -1)[:, :k]
    return _plain_values(q, e.int())


def _plain_norm(s):
    x, r = s["x"], s["residual"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS)
    return h, hf, rstd


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "norm_mx":
        h, hf, rstd = _plain_norm(s)
        q, e = _plain_parts(hf * rstd * s["weight"].float(), 8)
        out = {"y": _plain_values(q, e).to(torch.bfloat16)}
        return {**out, "h": h} if case["residual"] else out
    if op == "norm_train":
        h, hf, rstd = _plain_norm(s)
        w = s["weight"].float()
        hat = hf * rstd
        out = {"y": (hat * w).to(h.dtype)}
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - hat * (g * hat).mean(dim=1, keepdim=True))
        if case["residual"]:
            out["h"] = h
            dx = dx + s["dh"].float()
        out["dx"] = dx.to(h.dtype)
        out["dweight"] = (dy * hat).sum(dim=0).to(s["weight"].dtype)
        return out
    if op == "quantize":
        return {"values": _plain_values(*_plain_parts(s["x"].float(), case["bits"])).to(torch.bfloat16)}
    k = case["k"]
    w = _plain_decode(*s["weight"], case["wbits"], k)
    if op == "product":
        return {"c": (_plain_decode(*s["a"], case["bits"], k) @ w.t()).to(DTYPES[case["out"]])}
    x = _plain_values(*_plain_parts(s["x"].float(), case["bits"]))
    return {"c": (x @ w.t()).to(s["x"].dtype)}


# ---------------------------------------------------------------------------------- package's calls

def _calls(s):
    spt = _spt()
    case, op = s["case"], s["op"]
    if op == "norm_mx":
        if case["residual"]:
            q, h = spt.rms_norm_mx(s["x"], s["weight"], EPS, residual=s["residual"], bits=8)
            return {"y": spt.dequantize_mx(q, torch.bfloat16), "h": h}
        return {"y": spt.dequantize_mx(spt.rms_norm_mx(s["x"], s["weight"], EPS, bits=8), torch.bfloat16)}
    if op == "norm_train":
        if case["residual"]:
            y, h = spt.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
            dx, dw = spt.rms_norm_grad(s["dy"], h, s["weight"], EPS, dh=s["dh"])
            return {"y": y, "h": h, "dx": dx, "dweight": dw}
        y = spt.rms_norm(s["x"], s["weight"], EPS)
        dx, dw = spt.rms_norm_grad(s["dy"], s["x"], s["weight"], EPS)
        return {"y": y, "dx": dx, "dweight": dw}
    if op == "quantize":
        return {"values": spt.dequantize_mx(spt.quantize_mx(s["x"], case["bits"]), torch.bfloat16)}
    if op == "product":
        return {"c": spt.mx_matmul(s["a"], s["weight"], out_dtype=DTYPES[case["out"]])}
    return {"c": spt.mx_linear(s["x"], s["weight"], bits=case["bits"])}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------- 64 bits

def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_quantized(x, bits):
    """The definition: 2 to the floor of log2 of a block's largest magnitude, less the format's largest exponent; every
    value the nearest of the format's, the even code of two."""
    x = x.double()
    rows, k = x.shape
    n = (k + BLOCK - 1) // BLOCK
    full = torch.zeros((rows, n * BLOCK), dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, n, BLOCK)
    largest = full.abs().amax(dim=2, keepdim=True)
    _, exponent = torch.frexp(largest)  # largest = m * 2^exponent, 0.5 <= m < 1
    e = exponent - 1 - (2 if bits == 4 else 8)
    scale = torch.where(largest > 0, _power64(torch.clamp(e, min=-127)), 1.0)
    v = full / scale
    if bits == 4:
        values = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    else:
        codes = torch.arange(0, 127, dtype=torch.float64, device=x.device)  # 126: 448
        ex, mantissa = torch.div(codes, 8, rounding_mode="floor"), torch.remainder(codes, 8)
        values = torch.where(ex > 0, (8 + mantissa) * _power64(ex - 10), mantissa * 2.0 ** -9)
    mid = (values[1:] + values[:-1]) / 2
    mag = v.abs()
    low, high = torch.bucketize(mag, mid, right=False), torch.bucketize(mag, mid, right=True)
    at = torch.where(low % 2 == 0, low, high)  # they differ on a middle alone: the even one of the two
    q = torch.sign(v) * values[at] * scale
    return q.reshape(rows, n * BLOCK)[:, :k]


def _exact_decode(codes, e, bits, k):
    c = codes.long()
    if bits == 4:
        c = torch.stack([c % 16, c // 16], dim=2).reshape(c.shape[0], -1)[:, :k]
        table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=codes.device)
    else:
        table = []
        for i in range(128):
            table.append((i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10))
        table = torch.tensor(table + [-v for v in table], dtype=torch.float64, device=codes.device)
    scale = _power64(e.long() - 127)
    return table[c] * torch.repeat_interleave(scale, BLOCK, dim=1)[:, :k]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _exact_quantized(s["x"], case["bits"])}
    if op in ("product", "linear"):
        k = case["k"]
        w = _exact_decode(*s["weight"], case["wbits"], k)
        a = _exact_decode(*s["a"], case["bits"], k) if op == "product" else _exact_quantized(s["x"], case["bits"])
        return {"c": torch.mm(a, w.t())}
    x = s["x"].double()
    h = x
    if s["residual"] is not None:  # the sum is a tensor of the model: what is normalised is what is kept of it
        h = (x + s["residual"].double()).to(s["x"].dtype).double()
    w = s["weight"].double()
    n = h.shape[1]
    root = torch.sqrt(h.square().sum(dim=1, keepdim=True) / n + EPS)
    if op == "norm_mx":
        out = {"y": _exact_quantized(h / root * w, 8)}
    else:
        dy = s["dy"].double()
        g = dy * w
        dx = g / root - h * (g * h).sum(dim=1, keepdim=True) / (n * root ** 3)
        out = {"y": h / root * w, "dx": dx, "dweight": (dy * h / root).sum(dim=0)}
        if s["dh"] is not None:
            out["dx"] = dx + s["dh"].double()
    if s["residual"] is not None:
        out["h"] = h
    return out
