"""GPU tests of the microscaled tensors and their products against their definitions in 64 bits.

* Quantisation, its inverse and the layout are exact: equal bit for bit to the definition.
* Products of small integers with scales near 1 are exact in every step (each sum fits fp32, and every product lies within
  13 bits of the largest beside it): equal bit for bit, whichever kernel runs.
* Products of real values: an fp32 sum of k terms of total magnitude T is off by at most k 2^-23 T, whatever its order; a
  rounding to type t by at most u_t = eps_t / 2. With operands of 8 bits and a 16-bit result, the matrix instructions
  cut what lies 13 bits below the largest of the up to 16 products added at a time: each of those loses less than 2^-13
  of that largest one, so 16 of them less than 16 * 2^-13 of the 16's total magnitude: 2^-9 T.
"""
import copy
import pickle

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TINY = {F16: 2.0**-25, BF16: 2.0**-134, F32: 2.0**-150}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def power(e):
    """2^e for whole e in -1000 .. 1000, exact."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def levels(bits):
    """The format's values by code, in 64 bits; NaN at the 8-bit format's two codes for it."""
    if bits == 4:
        v = torch.tensor(E2M1, dtype=F64)
    else:
        c = torch.arange(128)
        e, m = c // 8, (c % 8).double()
        v = torch.where(e > 0, (8 + m) * power(e - 10), m * 2.0**-9)
        v[127] = float("nan")
    return torch.cat([v, -v]).cuda()


def scale_bytes(q):
    """[rows, blocks] of the layout's [rows / 64, blocks, 64]."""
    g, b, _ = q.scales.shape
    return q.scales.permute(0, 2, 1).reshape(g * 64, b)[: q.rows]


def codes_of(q):
    """One code per value, [rows, blocks * 32]."""
    c = q.codes.long()
    if q.bits == 4:
        c = torch.stack([c % 16, c // 16], dim=2).reshape(q.rows, -1)
    return c


def values(q):
    """The tensor's values by the formats' definition, in 64 bits, padding included."""
    s = scale_bytes(q).long().repeat_interleave(32, dim=1)
    v = levels(q.bits)[codes_of(q)] * power(s - 127)
    return torch.where(s == 255, float("nan"), v)


def quantized(x, bits):
    """Scale bytes [rows, blocks] and codes [rows, blocks * 32] by the definition."""
    x = x.to(F64)
    rows, k = x.shape
    n = (k + 127) // 128 * 4
    full = torch.zeros((rows, n * 32), dtype=F64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, n, 32)
    broken = ~torch.isfinite(full).all(dim=2)
    full = torch.where(broken[:, :, None], 0.0, full)
    top = full.abs().amax(dim=2)
    _, e = torch.frexp(top)
    s = torch.clamp(e.long() - 1 - (2 if bits == 4 else 8) + 127, min=0)
    s = torch.where(top > 0, s, 0)
    v = full * power(127 - s)[:, :, None]
    table = levels(bits)[: 8 if bits == 4 else 127]
    mid = (table[1:] + table[:-1]) / 2
    low, high = torch.bucketize(v.abs(), mid), torch.bucketize(v.abs(), mid, right=True)
    c = torch.where(low % 2 == 0, low, high) + torch.signbit(v) * (8 if bits == 4 else 128)
    c = torch.where(broken[:, :, None], 0, c)
    return torch.where(broken, 255, s), c.reshape(rows, n * 32)


def check_quantized(q, x):
    s, c = quantized(x, q.bits)
    assert torch.equal(scale_bytes(q).long(), s)
    assert torch.equal(codes_of(q), c)
    if q.rows % 64:  # rows that fill the last 64
        assert not q.scales[-1, :, q.rows % 64:].any()


def plain_codes(codes, bits, k):
    """Codes of one value each as a checkpoint holds them."""
    c = codes[:, :k].to(torch.uint8)
    if bits == 8:
        return c
    if k % 2:
        c = torch.cat([c, torch.full_like(c[:, :1], 9)], dim=1)  # a value behind the last, to be dropped
    return c[:, 0::2] | (c[:, 1::2] << 4)


def wide(shape, seed):
    """Normal values whose rows and columns differ by many powers of two."""
    g = gen(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return x * 2.0 ** torch.randint(-6, 7, (shape[0], 1), generator=g, device="cuda") * 2.0 ** torch.randint(-4, 5, (1, shape[1]), generator=g, device="cuda")


# -------------------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 31), (3, 32), (2, 33), (64, 128), (65, 127), (5, 129), (130, 500), (63, 512),
                                    (64, 513), (17, 4096), (257, 1030), (1, 8190), (1000, 2048)])
def test_quantize(rows, k, dtype, bits):
    x = wide((rows, k), rows * 7 + k).to(dtype)
    q = spt.quantize_mx(x, bits)
    assert q.shape == (rows, k) and q.dtype == dtype and q.bits == bits
    check_quantized(q, x)
    v = values(q)[:, :k]
    for out in (F16, BF16, F32):
        assert torch.equal(spt.dequantize_mx(q, out), v.to(out))


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_every_16_bit_value(bits):
    """Every bf16 and fp16 number as a block's largest and beside a larger one, ties and subnormal numbers among them."""
    for dtype in (BF16, F16):
        every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
        every = every[torch.isfinite(every)]
        x = every.repeat_interleave(32).view(-1, 32).clone()
        x[:, 1:] *= 0.37
        check_quantized(spt.quantize_mx(x, bits), x)
        x = every[torch.randperm(every.numel(), generator=gen(1), device="cuda")][: every.numel() // 128 * 128].view(-1, 128)
        check_quantized(spt.quantize_mx(x, bits), x)
        near = every.float().repeat_interleave(32).view(-1, 32) * torch.linspace(0.0, 1.0, 32, device="cuda")
        check_quantized(spt.quantize_mx(near, bits), near)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_ties(bits):
    """Middles of neighbouring values, in units of scales from the smallest on; a block's first value sets its scale."""
    table = levels(bits)[: 8 if bits == 4 else 127]
    mid = ((table[1:] + table[:-1]) / 2)
    for e in (-118, -60, 0, 60, 110):
        m = torch.cat([mid, -mid, table, -table]) * 2.0**e
        m = torch.nn.functional.pad(m, (0, -m.numel() % 31)).view(-1, 31).float()
        x = torch.cat([torch.full_like(m[:, :1], 2.0 ** (e + (2 if bits == 4 else 8))), m], dim=1)
        x[:, 1:] = torch.where(x[:, 1:].abs() >= 2 * x[:, :1], 0.0, x[:, 1:])
        check_quantized(spt.quantize_mx(x, bits), x)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_not_finite(bits, dtype):
    x = wide((70, 200), 3).to(dtype)
    x[0, 5], x[1, 40], x[69, 199], x[3, 64:96] = float("nan"), float("inf"), -float("inf"), 0.0
    q = spt.quantize_mx(x, bits)
    check_quantized(q, x)
    s = scale_bytes(q)
    assert s[0, 0] == s[1, 1] == s[69, 6] == 255 and (s == 255).sum() == 3 and s[3, 2] == 0
    v = spt.dequantize_mx(q, F32)
    assert torch.isnan(v[0, :32]).all() and torch.isnan(v[69, 192:]).all() and (v[3, 64:96] == 0).all()
    w = spt.quantize_mx(torch.ones((33, 200), device="cuda"), bits)
    for out in (BF16, F32):  # a NaN block makes its row's results NaN, and no other row's
        c = spt.mx_matmul(q, w, out)
        assert torch.isnan(c[[0, 1, 69]]).all() and torch.isfinite(c[2:69]).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,extra,offset", [(F16, 8, 0), (BF16, 3, 0), (F16, 0, 1), (BF16, 5, 3), (F32, 1, 1), (F32, 4, 0)])
def test_quantize_strides(dtype, extra, offset, bits):
    rows, k = 67, 333
    x = wide((rows, k), 11).to(dtype)
    buf = torch.full((rows * (k + extra) + offset,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:].view(rows, k + extra)[:, :k]
    v.copy_(x)
    q = spt.quantize_mx(v, bits)
    check_quantized(q, x)
    out = torch.full((rows * (k + extra) + offset,), 7.0, dtype=dtype, device="cuda")
    o = out[offset:].view(rows, k + extra)
    spt.dequantize_mx(q, out=o[:, :k])
    assert torch.equal(o[:, :k], values(q)[:, :k].to(dtype)) and (o[:, k:] == 7.0).all() and (out[:offset] == 7.0).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_dequantize_every_code_and_scale(bits):
    """All codes under all scales, to each type: subnormal results and infinities are the nearest of the type."""
    n = 16 if bits == 4 else 256
    codes = torch.arange(n, device="cuda").repeat(256, 1)
    s = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None].expand(256, -(-n // 32)).contiguous()
    q = spt.pack_mx(plain_codes(codes, bits, n), s, bits, n)
    v = values(q)[:, :n]
    for out in (F16, BF16, F32):
        got, want = spt.dequantize_mx(q, out), v.to(out)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, 0.0, 1e30, -1e30), torch.nan_to_num(want, 0.0, 1e30, -1e30))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,k", [(1, 1), (2, 3), (17, 259), (65, 510), (33, 513), (5, 770), (70, 1023)])
def test_dequantize_out(rows, k, dtype, bits):
    """Rows apart and off their size's alignment: the values, and nothing beside them."""
    q = int_operand(rows, k, bits, rows + k)
    buf = torch.full((rows * (k + 5) + 3,), 7.0, dtype=dtype, device="cuda")
    out = buf[3:].view(rows, k + 5)[:, :k]
    assert spt.dequantize_mx(q, out=out) is out
    want = values(q)[:, :k].to(F32).to(dtype)
    assert torch.equal(out, want) and torch.equal(spt.dequantize_mx(q, dtype), want)
    assert (buf[:3] == 7.0).all() and (buf[3:].view(rows, k + 5)[:, k:] == 7.0).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 32), (64, 128), (65, 95), (130, 500), (7, 1025)])
def test_pack(rows, k, bits):
    g = gen(rows + k)
    codes = torch.randint(0, 16 if bits == 4 else 256, (rows, k), generator=g, device="cuda")
    s = torch.randint(0, 256, (rows, -(-k // 32)), generator=g, device="cuda").to(torch.uint8)
    plain = plain_codes(codes, bits, k)
    q = spt.pack_mx(plain, s, bits, k)
    assert torch.equal(codes_of(q)[:, :k], codes) and not codes_of(q)[:, k:].any()
    assert torch.equal(scale_bytes(q)[:, : s.shape[1]], s) and not scale_bytes(q)[:, s.shape[1]:].any()
    wide_c = torch.full((rows, plain.shape[1] + 3), 255, dtype=torch.uint8, device="cuda")
    wide_s = torch.full((rows, s.shape[1] + 1), 255, dtype=torch.uint8, device="cuda")
    wide_c[:, 1:-2], wide_s[:, 1:] = plain, s
    again = spt.pack_mx(wide_c[:, 1:-2], wide_s[:, 1:], bits, k)
    assert torch.equal(again.codes, q.codes) and torch.equal(again.scales, q.scales)
    if bits == 8:
        typed = spt.pack_mx(plain.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu), 8, dtype=F16)
        assert torch.equal(typed.codes, q.codes) and typed.dtype == F16


# ------------------------------------------------------------------------------------------ products

def int_operand(rows, k, bits, seed, top=3, spread=2):
    """Small integers (those of e2m1) with scales of 2^-spread .. 2^spread."""
    g = gen(seed)
    c = torch.randint(0, 16, (rows, k), generator=g, device="cuda")
    v = torch.randint(-top, top + 1, (rows, k), generator=g, device="cuda").to(F32)
    s = torch.randint(127 - spread, 128 + spread, (rows, -(-k // 32)), generator=g, device="cuda").to(torch.uint8)
    if bits == 8:
        return spt.pack_mx(v.to(torch.float8_e4m3fn), s, 8, k)
    lut = torch.tensor([0, 2, 4, 5], device="cuda")
    c = lut[v.abs().long()] + (v < 0) * 8
    return spt.pack_mx(plain_codes(c, 4, k), s, 4, k)


def reference(a, b):
    x, y = values(a), values(b)
    return x @ y.t(), x.abs() @ y.abs().t()


FORMATS = [(8, 8), (4, 4), (8, 4)]
SHAPES = [(1, 1, 1), (1, 64, 128), (3, 5, 33), (2, 130, 31), (16, 16, 256), (17, 200, 300), (33, 63, 129), (64, 64, 64), (65, 127, 640),
          (127, 129, 257), (128, 128, 384), (130, 260, 1000), (256, 256, 512), (257, 511, 777), (300, 300, 100), (1, 1000, 4096),
          (5, 70, 9000), (40, 96, 12345), (100, 33, 5000), (513, 770, 1300), (4000, 2100, 300), (2049, 4099, 700)]


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_exact(m, n, k, fa, fb):
    a, b = int_operand(m, k, fa, m + k), int_operand(n, k, fb, n + k + 1)
    ref, _ = reference(a, b)
    for out in (F32, BF16, F16):
        assert torch.equal(spt.mx_matmul(a, b, out), ref.to(F32).to(out)), out


# By format and type these take, between them, every kernel with its sum whole and in parts, parts whose last one is a single step, more
# tiles than compute units, and 4-bit rows that end in half of a step. Sums stay below 2^24 units of 2^-2.
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", [(4668, 4694, 288), (2, 26, 7190), (605, 308, 21172), (1, 20, 161), (4447, 390, 214), (5874, 153, 8434),
                                   (582, 3899, 2602), (1398, 403, 33096), (1, 25, 1074), (20, 22, 419), (562, 577, 30747),
                                   (1, 21, 10692), (2461, 1707, 462), (1140, 3736, 16071), (5005, 971, 15845), (129, 5531, 20453)])
def test_matmul_every_kernel(m, n, k, fa, fb):
    a, b = int_operand(m, k, fa, m + k, spread=1), int_operand(n, k, fb, n + k + 1, spread=1)
    ref, _ = reference(a, b)
    for out in (F32, BF16, F16):
        buf = torch.full((m, n + 8), 7.0, dtype=out, device="cuda")  # what lies beside the result stays as it is
        spt.mx_matmul(a, b, out=buf[:, :n])
        assert torch.equal(buf[:, :n], ref.to(F32).to(out)), out
        assert (buf[:, n:] == 7.0).all()


def close(got, ref, total, k, dtype, fa):
    u = torch.finfo(dtype).eps / 2
    err = (k * 2.0**-23 + (2.0**-9 if fa == 8 and dtype != F32 else 0.0)) * total
    tol = err * (1 + u) + u * ref.abs() + TINY[dtype]
    off = (got.to(F64) - ref).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (16, 300, 2000), (40, 257, 4100), (130, 140, 8190), (300, 520, 640), (513, 1030, 1500)])
def test_matmul_real(m, n, k, fa, fb):
    a = spt.quantize_mx(wide((m, k), m).to(BF16), fa)
    b = spt.quantize_mx(wide((n, k), n + 1).to(F16), fb)
    ref, total = reference(a, b)
    for out in (F32, BF16, F16):
        got = spt.mx_matmul(a, b, out)
        fits = ref.abs() + 2.0**-8 * total < torch.finfo(out).max  # what its error can carry to infinity is left out
        close(torch.where(fits, got, 0.0), torch.where(fits, ref, 0.0), total, k, out, fa)
    # fp32 results of every format in 2-norm: k fp32 additions of random sign
    rel = ((spt.mx_matmul(a, b, F32).double() - ref).norm() / ref.norm()).item()
    assert rel < 1e-6


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("sa,sb", [(0, 254), (1, 250), (254, 0), (200, 10), (120, 134)])
def test_matmul_scales(fa, fb, sa, sb):
    """Scales at the ends of their range whose products are ordinary numbers."""
    m, n, k = 20, 70, 200
    a, b = int_operand(m, k, fa, 1, spread=0), int_operand(n, k, fb, 2, spread=0)
    a.scales[a.scales == 127] = sa
    b.scales[b.scales == 127] = sb
    ref, _ = reference(a, b)
    for out in (BF16, F16) if fa == 8 else (F32, BF16, F16):
        assert torch.equal(spt.mx_matmul(a, b, out), ref.to(F32).to(out))


@pytest.mark.parametrize("m,n,k", [(5, 77, 300), (70, 201, 1000), (300, 513, 260)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_matmul_out(m, n, k, dtype):
    for fa, fb in FORMATS:
        a, b = int_operand(m, k, fa, 5), int_operand(n, k, fb, 6)
        ref = reference(a, b)[0].to(F32).to(dtype)
        for extra, offset in ((0, 1), (3, 0), (5, 3)):
            buf = torch.full((m * (n + extra) + offset,), 7.0, dtype=dtype, device="cuda")
            o = buf[offset:].view(m, n + extra)
            got = spt.mx_matmul(a, b, out=o[:, :n])
            assert got.data_ptr() == o.data_ptr()
            assert torch.equal(o[:, :n], ref) and (o[:, n:] == 7.0).all() and (buf[:offset] == 7.0).all()


def test_empty():
    x = torch.empty((0, 100), device="cuda", dtype=BF16)
    q = spt.quantize_mx(x, 4)
    w = spt.quantize_mx(torch.ones((9, 100), device="cuda"), 4)
    assert spt.mx_matmul(q, w).shape == (0, 9) and spt.mx_matmul(w, q, F32).shape == (9, 0)
    assert spt.dequantize_mx(q).shape == (0, 100)
    none = spt.quantize_mx(torch.empty((5, 0), device="cuda", dtype=BF16), 8)
    other = spt.quantize_mx(torch.empty((7, 0), device="cuda", dtype=BF16), 8)
    for out in (BF16, F32):
        c = spt.mx_matmul(none, other, out)
        assert c.shape == (5, 7) and not c.any()
    assert spt.mx_linear(torch.empty((0, 100), device="cuda", dtype=F16), w).shape == (0, 9)


@pytest.mark.parametrize("bits,wbits", [(8, 8), (8, 4), (4, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_linear(bits, wbits, dtype):
    x, w = wide((37, 500), 1).to(dtype), spt.quantize_mx(wide((129, 500), 2), wbits)
    c = spt.mx_linear(x, w, bits)
    assert c.dtype == dtype
    assert torch.equal(c, spt.mx_matmul(spt.quantize_mx(x, bits), w, dtype))
    ref, total = reference(spt.quantize_mx(x, bits), w)
    fits = ref.abs() + 2.0**-8 * total < torch.finfo(dtype).max
    close(torch.where(fits, c, 0.0), torch.where(fits, ref, 0.0), total, 500, dtype, bits)


@pytest.mark.parametrize("fa,fb", FORMATS)
def test_same_bits_every_run(fa, fb):
    a, b = spt.quantize_mx(wide((60, 8190), 1), fa), spt.quantize_mx(wide((300, 8190), 2), fb)
    for out in (BF16, F32):
        first = spt.mx_matmul(a, b, out)
        for _ in range(5):
            assert torch.equal(spt.mx_matmul(a, b, out), first)


def test_copies_have_memory_of_their_own():
    for q in (spt.quantize_mx(wide((70, 300), 1).to(BF16), 4), int_operand(70, 300, 8, 1)):
        want = spt.dequantize_mx(q, F32)
        others = [copy.copy(q), copy.deepcopy(q), pickle.loads(pickle.dumps(q))]
        for other in others[1:]:
            assert other.codes_ptr != q.codes_ptr and other.codes_ptr == other.codes.data_ptr() and other.scales_ptr == other.scales.data_ptr()
        q.codes.zero_()
        assert torch.equal(spt.dequantize_mx(others[0], F32), torch.zeros_like(want))  # a shallow copy shares it
        for other in others[1:]:
            assert (other.bits, other.shape, other.dtype) == (q.bits, q.shape, q.dtype)
            assert torch.equal(spt.dequantize_mx(other, F32), want)


def test_streams():
    """Two calls at once with workspaces of their own, results used on their streams."""
    a, b = int_operand(20, 9000, 8, 1), int_operand(70, 9000, 4, 2)
    c, d = int_operand(30, 9000, 4, 3), int_operand(90, 9000, 4, 4)
    want = reference(a, b)[0].to(F32), reference(c, d)[0].to(F32)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        with torch.cuda.stream(s):
            x = spt.mx_matmul(a, b, F32)
        with torch.cuda.stream(t):
            y = spt.mx_matmul(c, d, F32)
        s.synchronize()
        t.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_two_graphs_replayed():
    """A quantised layer captured twice, replayed in turn with eager work between: no workspace is shared."""
    w = [spt.quantize_mx(wide((200, 6000), 5 + i), 4) for i in range(2)]
    x = [wide((9, 6000), 7 + i).to(BF16) for i in range(2)]
    eager = lambda i: spt.mx_linear(x[i], w[i], 8)  # noqa: E731
    eager(0)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(eager(i))
        graphs.append(g)
    for turn in range(4):
        for i in range(2):
            x[i].copy_(wide((9, 6000), 100 + 10 * turn + i).to(BF16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], eager(i))
