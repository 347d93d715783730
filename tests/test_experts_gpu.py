"""GPU tests of the experts' operators and the 4-bit products against their definitions in 64 bits.

Tolerances count roundings. A rounding to type t is off by at most u_t = eps_t / 2 relative to the
value (plus half the smallest subnormal). An fp32 sum of n terms of total magnitude T is off by at most
n * 2^-23 * T, whatever the order and whether the adder rounds to nearest (2^-24 each) or cuts off (2^-23
each). A product of two 16-bit values is exact in fp32; one of an fp32 weight with a 16-bit value is not,
and costs another 2^-24.
* Small-integer operands make every partial sum exact: those results must be equal bit for bit.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
TINY = {F16: 2.0**-25, BF16: 2.0**-134, F32: 2.0**-150}


def close(got, ref, total, n, dtype, extra=0.0):
    """|got - ref| <= n 2^-23 T + u|ref| (and the rounding acting on the sum's own error)."""
    u = torch.finfo(dtype).eps / 2
    err = (n * 2.0**-23 + extra) * total
    tol = err * (1 + u) + u * ref.abs() + TINY[dtype]
    bad = ~((got.to(F64) - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float(((got.to(F64) - ref).abs() / tol).max()))


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def ints(shape, dtype, seed, top=3):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").to(dtype)


def padded(t, extra, offset=0):
    """The same matrix with `extra` NaN elements between its rows, starting `offset` elements in."""
    r, c = t.shape[-2:]
    lead = t.shape[:-2]
    rows = int(np.prod(lead, dtype=np.int64)) * r
    buf = torch.full((rows * (c + extra) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[offset:].view(*lead, r, c + extra)[..., :c]
    v.copy_(t)
    return v


def ids_of(tokens, top_k, experts, seed, drop=0.2, dtype=torch.int64, skew=False):
    g = gen(seed)
    if skew:
        ids = (torch.rand((tokens, top_k), generator=g, device="cuda") ** 4 * experts).long().clamp_(max=experts - 1)
    else:
        ids = torch.randint(0, experts, (tokens, top_k), generator=g, device="cuda")
    lost = torch.rand((tokens, top_k), generator=g, device="cuda") < drop
    wrong = torch.where(torch.rand((tokens, top_k), generator=g, device="cuda") < 0.5, -1, experts)
    return torch.where(lost, wrong, ids).to(dtype)


def offsets_of(counts):
    return torch.tensor([0, *np.cumsum(counts).tolist()], dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------- sort

@pytest.mark.parametrize("tokens,top_k,experts", [
    (0, 2, 4), (1, 1, 1), (1, 8, 8), (63, 1, 3), (16, 4, 8), (65, 1, 64), (1000, 8, 127), (1024, 4, 128), (1024, 8, 128),
    (4096, 1, 255), (4097, 1, 255), (4097, 6, 64), (5000, 2, 1), (9001, 3, 1024), (100003, 3, 8), (300000, 1, 511), (1 << 17, 8, 256)])
@pytest.mark.parametrize("dtype,skew", [(torch.int64, False), (torch.int32, True)])
def test_sort(tokens, top_k, experts, dtype, skew):
    ids = ids_of(tokens, top_k, experts, tokens + experts, dtype=dtype, skew=skew)
    order = spt.sort_tokens(ids, experts)
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    slots = np.argsort(key, kind="stable")
    rows = np.empty_like(slots)
    rows[slots] = np.arange(slots.size)
    assert np.array_equal(order.slots.cpu().numpy(), slots)
    assert np.array_equal(order.rows.cpu().numpy(), rows.reshape(tokens, top_k))
    counts = np.bincount(key, minlength=experts + 1)
    assert np.array_equal(order.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts[:experts])]))


@pytest.mark.parametrize("value", [0, 6, -1, 7, 2**31, -(2**40), 2**32 + 3])
def test_sort_one_value(value):
    # everything in one group; 64-bit ids beyond 32 bits are dropped, not wrapped
    ids = torch.full((3000, 5), value, dtype=torch.int64, device="cuda")
    order = spt.sort_tokens(ids, 7)
    n = 15000
    assert torch.equal(order.slots, torch.arange(n, dtype=torch.int32, device="cuda"))
    inside = 0 <= value < 7
    want = [n if inside and e > value else 0 for e in range(8)]
    assert order.offsets.tolist() == want


# --------------------------------------------------------------------------- gather and combine

ROUTES = [(1, 1, 1, 8), (16, 2, 8, 4096), (7, 3, 5, 1), (33, 8, 16, 7), (129, 4, 9, 9), (50, 6, 64, 513), (64, 5, 3, 4097),
          (1030, 2, 8, 100), (3, 2, 4, 20000)]


def plain_combine(y, rows, kept, w):
    r = rows.long()
    on = (rows < kept)[:, :, None]
    t = torch.where(on, y.to(F64)[r], 0) * (w.to(F64)[:, :, None] if w is not None else 1)
    return t.sum(1), t.abs().sum(1)


@pytest.mark.parametrize("tokens,top_k,experts,width", ROUTES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gather_and_its_gradient(tokens, top_k, experts, width, dtype):
    order = spt.sort_tokens(ids_of(tokens, top_k, experts, width), experts)
    kept = int(order.offsets[-1])
    x = normal((tokens, width), dtype, 1)
    want = x[order.slots.long() // top_k].clone()
    want[kept:] = 0
    got = spt.gather_rows(x, order)
    assert torch.equal(got, want)
    # rows apart, an odd start; rows of `out` behind the last expert stay as they were
    out = torch.full((tokens * top_k, width + 3), 7.0, dtype=dtype, device="cuda")
    spt.gather_rows(padded(x, 5, 1), order, out=out[:, 1:1 + width])
    assert torch.equal(out[:kept, 1:1 + width], want[:kept])
    assert (out[kept:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 1 + width:] == 7).all()

    ds = normal((tokens * top_k, width), dtype, 2)
    ds[kept:] = float("nan")  # nothing behind the last expert is read
    ref, total = plain_combine(ds, order.rows, kept, None)
    close(spt.gather_rows_grad(ds, order), ref, total, top_k, dtype)
    close(spt.gather_rows_grad(padded(ds, 1, 3), order), ref, total, top_k, dtype)


@pytest.mark.parametrize("tokens,top_k,experts,width", ROUTES)
@pytest.mark.parametrize("dtype,wdtype", [(F16, F32), (BF16, F32), (F32, F32), (BF16, BF16), (F16, F16), (F16, None)])
def test_combine_and_its_gradients(tokens, top_k, experts, width, dtype, wdtype):
    order = spt.sort_tokens(ids_of(tokens, top_k, experts, width + 1), experts)
    kept = int(order.offsets[-1])
    y = normal((tokens * top_k, width), dtype, 3)
    y[kept:] = float("nan")
    w = normal((tokens, top_k), wdtype, 4) if wdtype else None
    ref, total = plain_combine(y, order.rows, kept, w)
    # the product's rounding is fused with the sum's; one more term for it where it is not
    close(spt.combine_rows(y, order, w), ref, total, top_k + 1, dtype)
    out = torch.full((tokens, width + 2), 7.0, dtype=dtype, device="cuda")
    spt.combine_rows(padded(y, 2, 1), order, w, out=out[:, :width])
    close(out[:, :width], ref, total, top_k + 1, dtype)
    assert (out[:, width:] == 7).all()

    dout = normal((tokens, width), dtype, 5)
    dy, dw = spt.combine_rows_grad(padded(dout, 1, 1), padded(y, 3), order, w)
    r, on = order.rows.long(), order.rows < kept
    want = dout.to(F64)[:, None, :] * (w.to(F64)[:, :, None] if w is not None else torch.ones_like(r)[:, :, None])
    want = torch.where(on[:, :, None], want, 0)
    close(dy[r], want, want.abs(), 1, dtype)
    if w is None:
        assert dw is None
    else:
        prod = torch.where(on[:, :, None], dout.to(F64)[:, None, :] * y.to(F64)[r], 0)
        close(dw, prod.sum(2), prod.abs().sum(2), width, wdtype)


def test_combine_keeps_infinities_to_their_tokens():
    order = spt.sort_tokens(torch.tensor([[0, 1], [1, 0], [2, 2]], device="cuda"), 3)
    y = torch.ones((6, 24), dtype=BF16, device="cuda")
    y[order.rows[0, 1].item(), 3] = float("inf")
    y[order.rows[1, 0].item(), 4] = float("nan")
    out = spt.combine_rows(y, order, torch.tensor([[1.0, -2.0], [0.5, 0.5], [0.0, 1.0]], device="cuda"))
    assert out[0, 3] == -float("inf") and out[1, 4].isnan() and out[2].eq(1).all()
    assert out.float().isfinite().sum() == 3 * 24 - 2


def test_rows_beyond_32_bits_of_bytes():
    # the sorted rows' last elements lie more than 2^32 bytes (and 2^31 elements) into the buffer
    tokens, width = 300_000, 7176
    order = spt.sort_tokens(torch.arange(tokens, device="cuda")[:, None] % 3, 3)
    x = (torch.arange(tokens, device="cuda") % 251).to(BF16)[:, None].expand(tokens, width).contiguous()
    got = spt.gather_rows(x, order)
    assert torch.equal(got[:, ::997].float(), (order.slots % 251).float()[:, None].expand(-1, 8))
    back = spt.combine_rows(got, order)
    assert torch.equal(back, x)


# ------------------------------------------------------------------------------- experts' products

def plain_grouped(mode, x, y, bounds, experts, n, k):
    rows = x.shape[0]
    x, y = x.to(F64), y.to(F64)
    if mode == "b":
        ref = torch.zeros((experts, n, k), dtype=F64, device="cuda")
        tot = torch.zeros_like(ref)
    else:
        ref = torch.zeros((rows, n if mode == "f" else k), dtype=F64, device="cuda")
        tot = torch.zeros_like(ref)
    for e in range(experts):
        s = slice(bounds[e], bounds[e + 1])
        if mode == "f":
            ref[s], tot[s] = x[s] @ y[e].t(), x[s].abs() @ y[e].abs().t()
        elif mode == "a":
            ref[s], tot[s] = x[s] @ y[e], x[s].abs() @ y[e].abs()
        else:
            ref[e], tot[e] = x[s].t() @ y[s], x[s].abs().t() @ y[s].abs()
    return ref, tot


def call_grouped(mode, x, y, off, out_dtype=None, tile=0):
    if mode == "f":
        return spt.grouped_matmul(x, y, off, out_dtype=out_dtype, tile=tile)
    if mode == "a":
        return spt.grouped_matmul_grad_a(x, y, off, tile=tile)
    return spt.grouped_matmul_grad_b(x, y, off, out_dtype=out_dtype, tile=tile)


def operands(mode, rows, experts, n, k, make):
    x = make((rows, k if mode == "f" else n), 11)
    y = make((rows, k) if mode == "b" else (experts, n, k), 12)
    return x, y


# counts per expert, rows behind the last one, n, k
GROUPS = [([1], 0, 1, 1), ([5], 0, 8, 8), ([0, 0, 0], 4, 16, 24), ([3, 0, 70, 1], 2, 33, 40), ([64, 128, 1, 127], 0, 64, 64),
          ([300, 0, 0, 513, 2], 7, 200, 136), ([129, 129], 1, 129, 65), ([17] * 70, 3, 72, 100), ([1000, 24], 0, 520, 1030),
          ([0] * 130 + [40], 0, 96, 264), ([2048], 0, 256, 512), ([257, 255, 600], 0, 511, 320)]


@pytest.mark.parametrize("counts,rest,n,k", GROUPS)
@pytest.mark.parametrize("mode", ["f", "a", "b"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_grouped_exact(counts, rest, n, k, mode, dtype):
    # integers up to 3 in magnitude: every sum is exact, fp32 outputs must be equal
    rows, experts = sum(counts) + rest, len(counts)
    off = offsets_of(counts)
    x, y = operands(mode, rows, experts, n, k, lambda s, seed: ints(s, dtype, seed))
    ref, _ = plain_grouped(mode, x, y, off.tolist(), experts, n, k)
    if mode != "b" and rest:
        x = x.clone()
        x[sum(counts):] = float("nan")  # rows behind the last expert are not part of any sum
    elif rest:
        x, y = x.clone(), y.clone()
        x[sum(counts):] = float("nan")
        y[sum(counts):] = float("inf")
    got = call_grouped(mode, x, y, off, F32)
    if mode == "a":  # dA comes in dC's type: the exact sum rounded once
        assert torch.equal(got, ref.to(dtype))
    else:
        assert torch.equal(got.to(F64), ref)
    # operands with rows apart (NaN between them) and, for odd distances, off 16 bytes
    for extra, start in ((8, 0), (3, 1)):
        got2 = call_grouped(mode, padded(x, extra, start), padded(y, extra, start), off, F32)
        assert torch.equal(got2, got), (extra, start)
    # every tile, and 16-bit outputs (the sums are below 2^24, rounded once)
    for tile in (32, 128, 256)[mode == "b":]:
        assert torch.equal(call_grouped(mode, x, y, off, F32, tile), got), tile
        assert torch.equal(call_grouped(mode, x, y, off, dtype, tile), got.to(dtype)), tile


@pytest.mark.parametrize("mode", ["f", "a", "b"])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, BF16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("counts,rest,n,k", [([700, 3, 0, 321], 10, 304, 456), ([9, 0, 14, 1, 30, 2, 0, 8], 0, 1001, 2048)])
def test_grouped_real(counts, rest, n, k, mode, dtype, out_dtype):
    rows, experts = sum(counts) + rest, len(counts)
    off = offsets_of(counts)
    x, y = operands(mode, rows, experts, n, k, lambda s, seed: normal(s, dtype, seed))
    ref, tot = plain_grouped(mode, x, y, off.tolist(), experts, n, k)
    got = call_grouped(mode, x, y, off, out_dtype)
    length = {"f": k, "a": n, "b": max(counts)}[mode]
    close(got, ref, tot, length, dtype if mode == "a" else out_dtype)
    assert torch.equal(call_grouped(mode, x, y, off, out_dtype), got)  # the same bits every time
    for tile in (32, 128, 256)[mode == "b":]:
        close(call_grouped(mode, x, y, off, out_dtype, tile), ref, tot, length, dtype if mode == "a" else out_dtype)


# tiles a workgroup takes one after another, each with one to three K-tiles: units, stores and loads of
# neighbouring tiles meet in every phase; empty experts in grad B are one K-tile of zeros
@pytest.mark.parametrize("mode", ["f", "a", "b"])
@pytest.mark.parametrize("length", [8, 64, 72, 136, 200])
@pytest.mark.parametrize("tile", [128, 256])
def test_grouped_many_tiles_of_short_sums(mode, length, tile):
    if mode == "b":
        counts, rest, n, k = [length, 0, length + 1, 3] * 4, 5, 1100, 2000
    else:
        counts, rest = [600, 0, 1, 257, 900, 0, 255], 300
        n, k = (2600, length) if mode == "f" else (length, 2600)
    off = offsets_of(counts)
    x, y = operands(mode, sum(counts) + rest, len(counts), n, k, lambda s, seed: ints(s, BF16, seed))
    ref, _ = plain_grouped(mode, x, y, off.tolist(), len(counts), n, k)
    for out_dtype in (F32, BF16):
        got = call_grouped(mode, x, y, off, out_dtype, tile)
        assert torch.equal(got, ref.to(got.dtype)), out_dtype


# the same with 32-row tiles, beyond the longest ring's sizes, aligned and not
@pytest.mark.parametrize("mode", ["f", "a"])
@pytest.mark.parametrize("length", [8, 72, 193, 200])
@pytest.mark.parametrize("width", [2600, 2605])
def test_grouped_many_small_tiles_of_short_sums(mode, length, width):
    counts, rest = [300, 0, 1, 129, 900, 0, 255], 300
    n, k = (width, length) if mode == "f" else (length, width)
    off = offsets_of(counts)
    x, y = operands(mode, sum(counts) + rest, len(counts), n, k, lambda s, seed: ints(s, F16, seed))
    ref, _ = plain_grouped(mode, x, y, off.tolist(), len(counts), n, k)
    for out_dtype in (F32, F16):
        got = call_grouped(mode, x, y, off, out_dtype, 32)
        assert torch.equal(got, ref.to(got.dtype)), out_dtype


# few rows and long sums: parts of the sum in planes, the last part cut by K or empty
@pytest.mark.parametrize("mode", ["f", "a"])
@pytest.mark.parametrize("counts,rest", [([1, 0, 1], 0), ([3], 2), ([0, 2, 40, 0, 1], 5), ([0, 0], 4), ([1] * 9, 0)])
@pytest.mark.parametrize("width,length", [(64, 1536), (146, 5556), (697, 2047), (1000, 4097), (33, 9001), (520, 1600)])
def test_grouped_long_sums_of_few_tiles(mode, counts, rest, width, length):
    n, k = (width, length) if mode == "f" else (length, width)
    rows, experts = sum(counts) + rest, len(counts)
    off = offsets_of(counts)
    x, y = operands(mode, rows, experts, n, k, lambda s, seed: ints(s, BF16, seed))
    ref, _ = plain_grouped(mode, x, y, off.tolist(), experts, n, k)
    if rest:
        x[sum(counts):] = float("nan")
    for tile in (0, 32):
        for out_dtype in (F32, BF16):
            got = call_grouped(mode, x, y, off, out_dtype, tile)
            assert torch.equal(got, ref.to(got.dtype)), (tile, out_dtype)
    got2 = call_grouped(mode, padded(x, 3, 1), padded(y, 3, 1), off, F32)
    assert torch.equal(got2, call_grouped(mode, x, y, off, F32))
    out = torch.full((rows, width + 7), 7.0, dtype=BF16, device="cuda")
    (spt.grouped_matmul if mode == "f" else spt.grouped_matmul_grad_a)(x, y, off, out=out[:, :width])
    kept = sum(counts)
    assert torch.equal(out[:kept, :width], ref[:kept].to(BF16)) and (out[kept:] == 7).all() and (out[:, width:] == 7).all()
    xr, yr = operands(mode, rows, experts, n, k, lambda s, seed: normal(s, F16, seed))
    ref, tot = plain_grouped(mode, xr, yr, off.tolist(), experts, n, k)
    close(call_grouped(mode, xr, yr, off, F16), ref, tot, length, F16)


# a little more than one round of 256 x 256 tiles over 256 compute units, the last tiles a row or a column wide
@pytest.mark.parametrize("mode", ["f", "a", "b"])
@pytest.mark.parametrize("length", [1024, 1101])
@pytest.mark.parametrize("width", [6016, 6273, 6145])
@pytest.mark.parametrize("counts,rest", [([1300, 0, 257, 900], 0), ([129, 128, 1281, 640, 1], 100), ([2700], 20)])
def test_grouped_second_round(mode, length, width, counts, rest):
    if mode == "b":
        counts, rest, n, k = [length, length + 65, length + 1, 2 * length][:len(counts) or 1], 7, 2056, width
        counts = counts if len(counts) > 1 else counts * 2
    else:
        n, k = (width, length) if mode == "f" else (length, width)
    rows, experts = sum(counts) + rest, len(counts)
    off = offsets_of(counts)
    x, y = operands(mode, rows, experts, n, k, lambda s, seed: ints(s, BF16, seed))
    ref, _ = plain_grouped(mode, x, y, off.tolist(), experts, n, k)
    for out_dtype in (F32, BF16):
        got = call_grouped(mode, x, y, off, out_dtype)
        assert torch.equal(got, ref.to(got.dtype)), out_dtype
        assert torch.equal(got, call_grouped(mode, x, y, off, out_dtype, 256)), out_dtype
    if mode != "b":
        out = torch.full((rows, width + 8), 7.0, dtype=BF16, device="cuda")
        (spt.grouped_matmul if mode == "f" else spt.grouped_matmul_grad_a)(x, y, off, out=out[:, :width])
        kept = sum(counts)
        assert torch.equal(out[:kept, :width], ref[:kept].to(BF16)) and (out[kept:] == 7).all() and (out[:, width:] == 7).all()


@pytest.mark.parametrize("mode", ["f", "a"])
@pytest.mark.parametrize("per", [5, 200])
def test_grouped_out_rows_left_as_they_were(mode, per):
    counts, rest, n, k = [per, 0, per + 1], 9, 72, 88
    rows, cols = sum(counts) + rest, n if mode == "f" else k
    off = offsets_of(counts)
    x, y = operands(mode, rows, 3, n, k, lambda s, seed: ints(s, BF16, seed))
    out = torch.full((rows, cols + 5), 7.0, dtype=BF16, device="cuda")
    view = out[:, 2:2 + cols]
    if mode == "f":
        spt.grouped_matmul(x, y, off, out=view)
    else:
        spt.grouped_matmul_grad_a(x, y, off, out=view)
    ref, _ = plain_grouped(mode, x, y, off.tolist(), 3, n, k)
    kept = sum(counts)
    assert torch.equal(view[:kept], ref[:kept].to(BF16))
    assert (out[kept:] == 7).all() and (out[:, :2] == 7).all() and (out[:, 2 + cols:] == 7).all()


@pytest.mark.parametrize("mode", ["f", "a", "b"])
def test_grouped_nonfinite_stays_in_place(mode):
    counts, n, k = [70, 60, 3], 40, 56
    off = offsets_of(counts)
    x, y = operands(mode, sum(counts), 3, n, k, lambda s, seed: ints(s, BF16, seed).abs() + 1)
    x = x.clone()
    x[75, 5], x[131, 7] = float("inf"), float("nan")
    got = call_grouped(mode, x, y, off, F32).float()
    bad = ~got.isfinite()
    want = torch.zeros_like(bad)
    if mode == "b":
        want[1, 5, :] = True
        want[2, 7, :] = True
        assert (got[1, 5] == float("inf")).all() and got[2, 7].isnan().all()
    else:
        want[75], want[131] = True, True
        assert (got[75] == float("inf")).all() and got[131].isnan().all()
    assert torch.equal(bad, want)


def test_grouped_strides_between_experts_and_empty_sizes():
    b = ints((4, 48, 64), F16, 3)
    wide = torch.full((4, 60, 72), float("nan"), dtype=F16, device="cuda")
    wide[:, 4:52, 8:] = b
    x = ints((50, 64), F16, 4)
    off = offsets_of([20, 0, 29])[[0, 1, 2, 2, 3]]
    ref, _ = plain_grouped("f", x, b, off.tolist(), 4, 48, 64)
    assert torch.equal(spt.grouped_matmul(x, wide[:, 4:52, 8:], off, out_dtype=F32).to(F64)[:49], ref[:49])
    # no rows, no columns, an empty sum, no experts
    z = offsets_of([0, 0])
    assert spt.grouped_matmul(x[:0], b[:2], z).shape == (0, 48)
    assert spt.grouped_matmul(x, b[:2, :0], z).shape == (50, 0)
    assert spt.grouped_matmul(x[:, :0], b[:2, :, :0], offsets_of([25, 25])).eq(0).all()
    assert spt.grouped_matmul(x, b[:0], offsets_of([])).eq(0).all()
    assert spt.grouped_matmul_grad_b(x[:0, :48], x[:0], z).eq(0).all()
    assert spt.grouped_matmul_grad_a(x[:, :0], b[:2, :0], offsets_of([25, 25])).eq(0).all()


def test_grouped_operands_beyond_32_bits():
    # rows whose elements lie beyond 2^31 elements (2^32 bytes) of A, C and dC
    rows, k, n = 600_000, 4096, 256
    a = torch.zeros((rows, k), dtype=BF16, device="cuda")
    mark = torch.tensor([0, 1, 255_999, 524_287, 524_288, 599_998, 599_999], device="cuda")
    a[mark] = ints((mark.numel(), k), BF16, 5)
    b = ints((2, n, k), BF16, 6)
    off = torch.tensor([0, 300_000, rows], dtype=torch.int32, device="cuda")
    c = spt.grouped_matmul(a, b, off, out_dtype=F32)
    for i, r in enumerate(mark.tolist()):
        assert torch.equal(c[r].to(F64), a[r].to(F64) @ b[int(r >= 300_000)].to(F64).t()), r
    assert int((c.abs().sum(1) > 0).sum()) <= mark.numel()
    dc = torch.zeros((rows, n), dtype=BF16, device="cuda")
    dc[mark] = ints((mark.numel(), n), BF16, 7)
    db = spt.grouped_matmul_grad_b(dc, a, off, out_dtype=F32)
    for e in range(2):
        m = mark[(mark >= 300_000) == bool(e)]
        assert torch.equal(db[e].to(F64), dc[m].to(F64).t() @ a[m].to(F64))
    da = spt.grouped_matmul_grad_a(dc, b, off)
    for r in mark.tolist():
        assert torch.equal(da[r], (dc[r].to(F64) @ b[int(r >= 300_000)].to(F64)).to(BF16)), r


# ----------------------------------------------------------------------------------- 4-bit weights

def w4_parts(shape, k, group, dtype, zeros, seed, exact=False):
    g = gen(seed)
    gs = -(-k // group)
    q = torch.randint(0, 16, (*shape, k), generator=g, device="cuda").to(torch.uint8)
    if exact:  # powers of two: the scaled sums stay exact
        s = (2.0 ** torch.randint(-2, 3, (*shape, gs), generator=g, device="cuda").float()).to(dtype)
    else:
        s = (0.01 + 0.02 * torch.rand((*shape, gs), generator=g, device="cuda")).to(dtype)
    z = torch.randint(0, 16, (*shape, gs), generator=g, device="cuda").to(torch.uint8) if zeros else None
    return q, s, z


def w4_dense(q, s, z, group):
    k = q.shape[-1]
    at = torch.arange(k, device="cuda") // group
    zz = z.to(F64)[..., at] if z is not None else 8.0
    return (q.to(F64) - zz) * s.to(F64)[..., at]


W4_SHAPES = [(1, 1, 1), (1, 16, 128), (2, 17, 31), (5, 100, 33), (16, 64, 256), (17, 48, 1000), (1, 1024, 4096), (33, 40, 520),
             (64, 130, 384), (65, 257, 129), (200, 96, 640), (3, 2056, 8190), (16, 16400, 256),
             # one shape for each kernel the choice goes to as the output grows, with blocks of K that K cuts
             (2, 4160, 200), (15, 17500, 2201), (40, 8000, 303), (130, 9000, 300), (300, 8001, 517), (70, 24000, 120),
             (520, 8200, 261), (301, 1030, 4097)]


@pytest.mark.parametrize("rows,n,k", W4_SHAPES)
@pytest.mark.parametrize("dtype,group,zeros", [(F16, 32, False), (F16, 64, True), (F16, 128, True), (BF16, 32, True),
                                              (BF16, 64, False), (BF16, 128, False), (BF16, 128, True)])
def test_w4_exact_and_real(rows, n, k, dtype, group, zeros):
    q, s, z = w4_parts((n,), k, group, dtype, zeros, rows + n + k, exact=True)
    w = spt.pack_w4(q, s, z, group)
    x = ints((rows, k), dtype, 21, top=2)
    ref = x.to(F64) @ w4_dense(q, s, z, group).t()  # at most 2 * 15 * 4 * 8190 in quarters: exact in fp32
    assert torch.equal(spt.w4_matmul(x, w, out_dtype=F32).to(F64), ref)
    assert torch.equal(spt.w4_matmul(padded(x, 3, 1), w, out_dtype=F32).to(F64), ref)
    assert torch.equal(spt.w4_matmul(padded(x, 8, 0), w), ref.to(dtype))

    q, s, z = w4_parts((n,), k, group, dtype, zeros, rows + n + k + 1)
    x = normal((rows, k), dtype, 22)
    d = w4_dense(q, s, z, group)
    got = spt.w4_matmul(x, spt.pack_w4(q, s, z, group))
    # group sums and their sum: one fp32 rounding a term, one more per scale
    close(got, x.to(F64) @ d.t(), x.to(F64).abs() @ d.abs().t(), k + 2, dtype)


@pytest.mark.parametrize("counts,rest", [([1, 0, 2, 0], 0), ([3, 0, 20, 1, 64, 0, 7, 9], 5), ([0, 0], 3), ([70, 130, 0, 1], 0),
                                        ([1] * 70, 2), ([29, 31, 0, 40] * 5, 1), ([100, 0, 130, 1] * 5, 9)])
@pytest.mark.parametrize("n,k", [(48, 384), (257, 1023), (2000, 128), (1000, 2100)])
@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, False), (F16, 32, True)])
def test_w4_experts(counts, rest, n, k, dtype, group, zeros):
    e, rows = len(counts), sum(counts) + rest
    off = offsets_of(counts)
    q, s, z = w4_parts((e, n), k, group, dtype, zeros, n + k, exact=True)
    w = spt.pack_w4(q, s, z, group)
    x = ints((rows, k), dtype, 23, top=2)
    ref = torch.zeros((rows, n), dtype=F64, device="cuda")
    for i in range(e):
        part = slice(int(off[i]), int(off[i + 1]))
        ref[part] = x[part].to(F64) @ w4_dense(q[i], s[i], z[i] if zeros else None, group).t()
    x[sum(counts):] = float("nan")
    assert torch.equal(spt.w4_matmul(x, w, off, out_dtype=F32).to(F64), ref)
    out = torch.full((rows, n + 1), 7.0, dtype=F32, device="cuda")
    spt.w4_matmul(x, w, off, out=out[:, :n])
    assert torch.equal(out[:sum(counts), :n].to(F64), ref[:sum(counts)])
    assert (out[sum(counts):] == 7).all() and (out[:, n] == 7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [1, 20])
def test_w4_nonfinite_inputs_and_zero_weights(dtype, rows):
    n, k, group = 64, 512, 64
    q, s, z = w4_parts((n,), k, group, dtype, True, 31)
    at = torch.arange(k, device="cuda") // group
    q[5] = z[5][at]  # a column whose weights are all zero
    x = normal((rows, k), dtype, 32, 100.0)
    w = spt.pack_w4(q, s, z, group)
    assert (spt.w4_matmul(x, w, out_dtype=F32)[:, 5] == 0).all()
    x[0, 77] = float("inf")
    got = spt.w4_matmul(x, w, out_dtype=F32)
    sign = q[:, 77].float() - z[:, 77 // group].float()
    want = torch.where(sign == 0, float("nan"), torch.where(sign > 0, float("inf"), -float("inf")))
    assert torch.equal(got[0].isnan(), want.isnan()) and torch.equal(got[0].nan_to_num(1), want.nan_to_num(1))
    assert got[1:].isfinite().all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_w4_subnormal_and_large_inputs(dtype):
    n, k = 32, 256
    q, s, z = w4_parts((n,), k, 128, dtype, False, 33)
    for scale in (2.0**-20 if dtype == F16 else 2.0**-100, 1000.0 if dtype == F16 else 2.0**100):
        x = normal((3, k), dtype, 34, scale)
        d = w4_dense(q, s, z, 128)
        close(spt.w4_matmul(x, spt.pack_w4(q, s, z, 128), out_dtype=F32), x.to(F64) @ d.t(),
              x.to(F64).abs() @ d.abs().t(), k + 2, F32)


def test_w4_packs_of_strided_and_empty_tensors():
    q, s, z = w4_parts((24,), 96, 32, F16, True, 35, exact=True)
    x = ints((4, 96), F16, 36)
    want = spt.w4_matmul(x, spt.pack_w4(q, s, z, 32))
    qt, st, zt = (t.t().contiguous().t() for t in (q, s, z))
    assert torch.equal(spt.w4_matmul(x, spt.pack_w4(qt + 16 * 7, st, zt, 32)), want)  # the low four bits count
    assert spt.w4_matmul(x, spt.pack_w4(q[:0], s[:0], z[:0], 32)).shape == (4, 0)
    assert spt.w4_matmul(x[:, :0], spt.pack_w4(q[:, :0], s[:, :0], z[:, :0], 32)).eq(0).all()
    assert spt.w4_matmul(x[:0], spt.pack_w4(q, s, z, 32)).shape == (0, 24)


# -------------------------------------------------------------------------------------- together

def routed_reference(x, b, ids, w):
    out = torch.zeros((x.shape[0], b.shape[1]), dtype=F64, device="cuda")
    for j in range(ids.shape[1]):
        for e in range(b.shape[0]):
            m = (ids[:, j] == e).nonzero()[:, 0]
            out = out.index_add(0, m, (x[m] @ b[e].t()) * w[m, j, None])
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,top_k,experts,n,k", [(1, 2, 4, 24, 16), (40, 3, 7, 65, 72), (300, 2, 4, 128, 250)])
def test_routed_layer_and_its_gradients(tokens, top_k, experts, n, k, dtype):
    ids = ids_of(tokens, top_k, experts, 41)
    x = normal((tokens, k), dtype, 42).requires_grad_()
    b = normal((experts, n, k), dtype, 43, k**-0.5).requires_grad_()
    w = torch.rand((tokens, top_k), generator=gen(44), device="cuda").requires_grad_()
    dout = normal((tokens, n), dtype, 45)
    out = spt.routed_matmul(x, b, ids, w)
    gx, gb, gw = torch.autograd.grad(out, (x, b, w), dout)
    ref_in = [t.detach().to(F64).requires_grad_() for t in (x, b, w)]
    ref = routed_reference(ref_in[0], ref_in[1], ids, ref_in[2])
    rx, rb, rw = torch.autograd.grad(ref, ref_in, dout.to(F64))
    mag = [t.detach().to(F64).abs().requires_grad_() for t in (x, b, w)]
    tot = routed_reference(*[mag[0], mag[1], ids, mag[2]])
    tx, tb, tw = torch.autograd.grad(tot, mag, dout.to(F64).abs())
    # two or three roundings to 16 bits on the way (the experts' rows, their gradients), each relative to
    # terms whose magnitudes add up to the total
    u = torch.finfo(dtype).eps / 2
    close(out, ref.detach(), tot.detach(), k + top_k + 1, dtype, extra=2 * u)
    close(gx, rx, tx, n + top_k + 1, dtype, extra=3 * u)
    close(gb, rb, tb, tokens + 1, dtype, extra=2 * u)
    close(gw, rw, tw, n + k, F32, extra=2 * u)


def test_gradients_match_differences():
    # every operator is linear in each input, so a difference along a direction equals the gradient's
    # product with it; small integers and power-of-two weights make both sides exact
    tokens, top_k, experts, n, k = 60, 2, 5, 48, 40
    ids = ids_of(tokens, top_k, experts, 51)
    order = spt.sort_tokens(ids, experts)
    off = order.offsets
    x, b = ints((tokens, k), BF16, 52, 2), ints((experts, n, k), BF16, 53, 2)
    w = (2.0 ** torch.randint(-1, 2, (tokens, top_k), generator=gen(54), device="cuda")).to(F32)
    rows = spt.gather_rows(x, order)
    dc = ints((tokens * top_k, n), BF16, 55, 2)

    def dot(p, q):
        return float((p.to(F64) * q.to(F64)).sum())
    h = ints(rows.shape, BF16, 56, 1)
    kept = torch.arange(rows.shape[0], device="cuda")[:, None] < off[-1]
    f = lambda a_, b_: dot(spt.grouped_matmul(a_, b_, off, out_dtype=F32), dc)  # noqa: E731
    assert f(rows + h, b) - f(rows, b) == dot(spt.grouped_matmul(h, b, off, out_dtype=F32), dc)
    da = torch.where(kept, spt.grouped_matmul_grad_a(dc, b, off).to(F64), 0)
    ref = plain_grouped("a", dc, b, off.tolist(), experts, n, k)[0]
    assert torch.equal(da, ref.to(BF16).to(F64))
    hb = ints(b.shape, BF16, 57, 1)
    assert f(rows, b + hb) - f(rows, b) == dot(spt.grouped_matmul_grad_b(dc, rows, off, out_dtype=F32), hb)
    # gather and combine
    hx = ints(x.shape, BF16, 58, 1)
    ds = ints(rows.shape, BF16, 59, 2)
    g = lambda v: dot(spt.gather_rows(v, order), ds)  # noqa: E731
    assert g(x + hx) - g(x) == dot(spt.gather_rows_grad(ds, order), hx)
    y, dout = ints((tokens * top_k, n), F32, 60, 2), ints((tokens, n), F32, 61, 2)
    hy, hw = ints(y.shape, F32, 62, 1), ints(w.shape, F32, 63, 1)
    c = lambda y_, w_: dot(spt.combine_rows(y_, order, w_), dout)  # noqa: E731
    dy, dw = spt.combine_rows_grad(dout, y, order, w)
    assert c(y + hy, w) - c(y, w) == dot(dy, hy)
    assert c(y, w + hw) - c(y, w) == dot(dw, hw)


def test_autograd_of_single_operators_with_broadcast_gradients():
    order = spt.sort_tokens(ids_of(20, 2, 3, 71), 3)
    kept = int(order.offsets[-1])
    x = ints((20, 16), F16, 72).requires_grad_()
    spt.gather_rows(x, order).sum().backward()  # an expanded gradient of ones
    assert torch.equal(x.grad, (order.rows < kept).sum(1, keepdim=True).to(F16).expand(20, 16))
    a, b = ints((40, 16), F16, 73).requires_grad_(), ints((3, 8, 16), F16, 74).requires_grad_()
    spt.grouped_matmul(a, b, order.offsets).sum().backward()
    ones = torch.ones((40, 8), dtype=F16, device="cuda")
    assert torch.equal(a.grad, spt.grouped_matmul_grad_a(ones, b, order.offsets))
    assert torch.equal(b.grad, spt.grouped_matmul_grad_b(ones, a, order.offsets))
    a.grad = None
    spt.grouped_matmul(a, b.detach(), order.offsets, out_dtype=F32).t().mul(2).sum().backward()  # fp32, transposed
    assert torch.equal(a.grad, spt.grouped_matmul_grad_a(2 * ones, b, order.offsets))
    y = ints((40, 8), F32, 75).requires_grad_()
    w = torch.ones((20, 2), device="cuda", requires_grad=True)
    spt.combine_rows(y, order, w).sum().backward()
    assert torch.equal(w.grad, torch.where(order.rows < kept, y.detach().sum(1)[order.rows.long()], 0))


def test_routed_layer_of_four_bit_experts():
    tokens, top_k, experts, n, k = 24, 2, 6, 80, 192
    ids = ids_of(tokens, top_k, experts, 81)
    q, s, z = w4_parts((experts, n), k, 64, BF16, True, 82, exact=True)
    x, w = ints((tokens, k), BF16, 83, 1), torch.rand((tokens, top_k), generator=gen(84), device="cuda")
    got = spt.routed_matmul(x, spt.pack_w4(q, s, z, 64), ids, w)
    d = w4_dense(q, s, z, 64)
    ref, tot = (routed_reference(f(x.to(F64)), f(d), ids, w.to(F64)) for f in (lambda t: t, torch.abs))
    close(got, ref, tot, top_k + 1, BF16, extra=2.0**-8)


# ------------------------------------------------------------------------------ streams and graphs

def step(x, b, ids, w, dout, q4, order_experts):
    order = spt.sort_tokens(ids, order_experts)
    rows = spt.gather_rows(x, order)
    y = spt.grouped_matmul(rows, b, order.offsets)
    out = spt.combine_rows(y, order, w)
    dy, dw = spt.combine_rows_grad(dout, y, order, w)
    drows = spt.grouped_matmul_grad_a(dy, b, order.offsets)
    db = spt.grouped_matmul_grad_b(dy, rows, order.offsets)
    dx = spt.gather_rows_grad(drows, order)
    y4 = spt.w4_matmul(rows, q4, order.offsets)
    return [out, dw, db, dx, y4, order.slots]


def step_inputs(tokens, seed, odd):
    experts, n, k = 5, 72 + odd, 200 + odd  # odd sizes go through padded copies
    ids = ids_of(tokens, 2, experts, seed)
    x, b = normal((tokens, k), BF16, seed + 1), normal((experts, n, k), BF16, seed + 2)
    w = torch.rand((tokens, 2), generator=gen(seed + 3), device="cuda")
    q, s, z = w4_parts((experts, n), k, 32, BF16, True, seed + 5)
    return [x, b, ids, w, normal((tokens, n), BF16, seed + 4), spt.pack_w4(q, s, z, 32), experts]


@pytest.mark.parametrize("odd", [0, 1])
def test_captured_steps_replay_to_the_eager_bits(odd):
    # two graphs of different sizes (4100 tokens: a sort over several workgroups), replayed in turn between
    # eager steps; inputs change in place between replays
    cases = [step_inputs(4200, 91, odd), step_inputs(33, 95, odd)]
    for c in cases:
        step(*c)
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*c)
        graphs.append((g, out))
    for rep in range(4):
        for (g, out), c in zip(graphs, cases):
            c[0].copy_(normal(c[0].shape, BF16, 100 + rep))
            c[2].copy_(ids_of(c[2].shape[0], 2, 5, 200 + rep))
            want = step(*c)
            torch.cuda.synchronize()
            for o in out:
                o.zero_()
            g.replay()
            step(*cases[0])
            torch.cuda.synchronize()
            for o, e in zip(out, want):
                assert torch.equal(o, e), rep


def test_captured_autograd_step():
    # autograd's own way: warmed up on the capture's kind of stream, and no eager graph of the leaves alive
    x, b = normal((70, 96), BF16, 161).requires_grad_(), normal((5, 130, 96), BF16, 162).requires_grad_()
    w = torch.rand((70, 2), device="cuda").requires_grad_()
    ids, dout = ids_of(70, 2, 5, 163), normal((70, 130), BF16, 164)

    def train():
        return torch.autograd.grad(spt.routed_matmul(x, b, ids, w), (x, b, w), dout)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            train()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = train()
    for rep in range(3):
        with torch.no_grad():
            x.copy_(normal(x.shape, BF16, 170 + rep))
            dout.copy_(normal(dout.shape, BF16, 180 + rep))
        g.replay()
        torch.cuda.synchronize()
        for a, e in zip(got, train()):
            assert torch.equal(a, e), rep


def test_side_streams_at_once():
    cases = [step_inputs(900, 110 + i, i & 1) for i in range(4)]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append([step(*c) for _ in range(3)])
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        for r in runs:
            for a, e in zip(r, w):
                assert torch.equal(a, e)


# ------------------------------------------------------------------------------- contents gone wrong

@pytest.mark.parametrize("off", [[5, 2, 40, 10], [-7, 30, 30, 1000], [0, 0, 0, -1], [60, 50, 40, 30],
                                 [2**31 - 1, -(2**31), 7, 2**30]])
def test_wrong_offsets_stay_inside_the_operands(off):
    # offsets are clamped to the operands: the results mean nothing, but nothing else is touched
    rows, n, k = 50, 72, 88
    guard = 64
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, b = ints((rows, k), BF16, 131), ints((3, n, k), BF16, 132)
    dc = ints((rows, n), BF16, 133)
    q, s, z = w4_parts((3, n), k, 32, BF16, True, 134)
    w = spt.pack_w4(q, s, z, 32)
    for tile in (32, 128, 256):
        c = torch.full((rows + 2 * guard, n), 7.0, dtype=BF16, device="cuda")
        spt.grouped_matmul(x, b, offsets, out=c[guard:-guard], tile=tile)
        a = torch.full((rows + 2 * guard, k), 7.0, dtype=BF16, device="cuda")
        spt.grouped_matmul_grad_a(dc, b, offsets, out=a[guard:-guard], tile=tile)
        for t in (c, a):
            assert (t[:guard] == 7).all() and (t[-guard:] == 7).all()
        if tile != 32:
            assert spt.grouped_matmul_grad_b(dc, x, offsets, tile=tile).shape == (3, n, k)
    c = torch.full((rows + 2 * guard, n), 7.0, dtype=BF16, device="cuda")
    spt.w4_matmul(x, w, offsets, out=c[guard:-guard])
    assert (c[:guard] == 7).all() and (c[-guard:] == 7).all()


def test_wrong_positions_stay_inside_the_operands():
    order = spt.sort_tokens(ids_of(20, 2, 3, 141), 3)
    order.rows.copy_(torch.tensor([-5, 1000, 2**31 - 1, -(2**31), 39, 40, 3, 3] * 5, dtype=torch.int32).view(20, 2))
    x = ints((20, 24), F16, 142)
    out = torch.full((40 + 128, 24), 7.0, dtype=F16, device="cuda")
    spt.gather_rows(x, order, out=out[64:-64])
    assert (out[:64] == 7).all() and (out[-64:] == 7).all()
    y = ints((40, 24), F16, 143)
    assert spt.combine_rows(y, order).shape == (20, 24)
    dy, dw = spt.combine_rows_grad(x, y, order, torch.ones((20, 2), device="cuda"))
    assert dy.shape == y.shape and dw[0].eq(0).all()


def test_no_slots_and_no_tokens():
    order = spt.sort_tokens(torch.zeros((5, 0), dtype=torch.int64, device="cuda"), 3)
    x = ints((5, 16), F16, 151)
    assert order.offsets.eq(0).all() and spt.gather_rows(x, order).shape == (0, 16)
    assert spt.combine_rows(x[:0], order).eq(0).all() and spt.gather_rows_grad(x[:0], order).shape == (5, 16)
    order = spt.sort_tokens(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 3)
    assert spt.combine_rows(x[:0], order, torch.zeros((0, 2), device="cuda")).shape == (0, 16)
    b = ints((3, 8, 16), F16, 152)
    assert spt.routed_matmul(x[:0], b, torch.zeros((0, 2), dtype=torch.int64, device="cuda")).shape == (0, 8)
    ids = torch.full((5, 2), -1, dtype=torch.int64, device="cuda")  # every slot dropped
    w = torch.ones((5, 2), device="cuda", requires_grad=True)
    out = spt.routed_matmul(x, b, ids, w)
    out.sum().backward()
    assert out.eq(0).all() and w.grad.eq(0).all()


# --------------------------------------------------------------------------------------- refusals

def test_refusals_of_shapes_and_layouts():
    order = spt.sort_tokens(ids_of(8, 2, 3, 121), 3)
    off = order.offsets
    x, b = ints((8, 16), BF16, 122), ints((3, 24, 16), BF16, 123)
    rows = spt.gather_rows(x, order)
    q, s, z = w4_parts((3, 24), 16, 32, BF16, False, 124)
    w3, w1 = spt.pack_w4(q, s, None, 32), spt.pack_w4(q[0], s[0], None, 32)
    bad = [
        lambda: spt.sort_tokens(ids_of(8, 2, 3, 1)[None], 3),
        lambda: spt.gather_rows(x[:7], order), lambda: spt.gather_rows(x.t().contiguous().t(), order),
        lambda: spt.gather_rows(x[:1].expand(8, 16), order), lambda: spt.gather_rows(x, order, out=rows[:, :8]),
        lambda: spt.gather_rows(x, order, out=rows.float()), lambda: spt.combine_rows(x, order),
        lambda: spt.combine_rows(rows, order, torch.ones((8, 3), device="cuda")),
        lambda: spt.combine_rows_grad(x.float(), rows, order), lambda: spt.combine_rows_grad(x[:, :8], rows, order),
        lambda: spt.grouped_matmul(rows, b[:, :, :8], off), lambda: spt.grouped_matmul(rows, b, off.long()),
        lambda: spt.grouped_matmul(rows, b, off[:-1]), lambda: spt.grouped_matmul(rows, b.half(), off),
        lambda: spt.grouped_matmul(rows, b[0], off), lambda: spt.grouped_matmul(rows, b[:1].expand(3, 24, 16), off),
        lambda: spt.grouped_matmul(rows, b, off, out=rows), lambda: spt.grouped_matmul(rows, b, off.cpu()),
        lambda: spt.grouped_matmul_grad_a(rows, b, off), lambda: spt.grouped_matmul_grad_b(rows, x, off),
        lambda: spt.w4_matmul(x, w3), lambda: spt.w4_matmul(x, w1, off), lambda: spt.w4_matmul(x.half(), w1),
        lambda: spt.w4_matmul(x[:, :8], w1), lambda: spt.w4_matmul(x.clone().requires_grad_(), w1),
        lambda: spt.pack_w4(q, s, None, 48), lambda: spt.pack_w4(q, s[:, :, :0], None, 32),
        lambda: spt.pack_w4(q, s, s.byte()[:, :2], 32), lambda: spt.routed_matmul(x, w1, ids_of(8, 2, 3, 2)),
        lambda: spt.routed_matmul(x, b, ids_of(7, 2, 3, 2)),
        lambda: spt.gather_rows(x.clone().requires_grad_(), order, out=rows.clone()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    with pytest.raises(spt.GemmError):
        spt.sort_tokens(ids_of(8, 2, 3, 3), 0)
    with pytest.raises(spt.GemmError):
        spt.sort_tokens(ids_of(8, 2, 3, 3), 1025)
    with pytest.raises(TypeError):
        spt.grouped_matmul(rows, b, off, out_dtype=torch.float64)
    assert torch.equal(spt.gather_rows(x, order), rows)  # nothing above touched anything
