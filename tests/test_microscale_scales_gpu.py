"""GPU tests of products whose scales reach the ends of their bytes, against 64 bits.

Powers of two are exact, so small integers at any scale whose products are ordinary numbers give the definition's bits. Where scales
of every size meet, an fp32 sum of k terms of total magnitude T is off by at most k 2^-23 T; a product below 2^-126, which fp32
holds with fewer bits, may count as zero: k 2^-126 more. Results are compared where no sum of some of the terms can pass fp32's end (T < 2^127).
16-bit results of 8-bit operands: 2^-9 T more, the matrix instructions' cut at 13 bits below the largest of 16 products.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402
from test_microscale_gpu import gen, int_operand, plain_codes, reference, scale_bytes, values  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
FORMATS = [(8, 8), (8, 4), (4, 4)]
# few rows, tiles of 32, 64 and 128 rows, a sum in parts, tiles of 256
SHAPES = [(3, 70, 200), (20, 100, 1500), (40, 200, 640), (100, 300, 300), (300, 1500, 1000), (5, 20, 9000), (700, 900, 2000)]


def set_scales(q, s):
    """Scale bytes [rows, blocks that hold values]."""
    g, b, _ = q.scales.shape
    full = torch.zeros((g * 64, b), dtype=torch.uint8, device="cuda")
    full[: s.shape[0], : s.shape[1]] = s
    q.scales.copy_(full.view(g, 64, b).permute(0, 2, 1))
    assert torch.equal(scale_bytes(q), full[: q.rows])


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("sa,sb", [(0, 254), (254, 0), (1, 250), (9, 245), (10, 244), (11, 243), (246, 8), (247, 7), (245, 9), (63, 191), (64, 190)])
def test_ordinary_products(m, n, k, sa, sb, fa, fb):
    """All blocks at one end, and only one row's and one column's."""
    for rows, cols in ((slice(None), slice(None)), (slice(m // 2, m // 2 + 1), slice(None)), (slice(None), slice(n // 3, n // 3 + 1))):
        a, b = int_operand(m, k, fa, m + 1, spread=0), int_operand(n, k, fb, n + 2, spread=0)
        blocks = -(-k // 32)
        x, y = torch.full((m, blocks), 127, device="cuda", dtype=torch.uint8), torch.full((n, blocks), 127, device="cuda", dtype=torch.uint8)
        x[rows], y[cols] = sa, sb
        set_scales(a, x)
        set_scales(b, y)
        ref, total = reference(a, b)
        ordinary = (total < 2.0**100) & ((ref == 0) | (ref.abs() > 2.0**-100))
        got = spt.mx_matmul(a, b, F32)
        assert ordinary.any() and torch.equal(got[ordinary], ref.to(F32)[ordinary])


def mixed(rows, k, bits, seed, sizes):
    """Any codes of the format but NaN, each block's scale one of `sizes`."""
    g = gen(seed)
    if bits == 4:
        c = torch.randint(0, 16, (rows, k), generator=g, device="cuda")
    else:
        c = torch.randint(0, 127, (rows, k), generator=g, device="cuda") + 128 * torch.randint(0, 2, (rows, k), generator=g, device="cuda")
    t = torch.tensor(sizes, device="cuda", dtype=torch.uint8)
    s = t[torch.randint(0, len(sizes), (rows, -(-k // 32)), generator=g, device="cuda")]
    return spt.pack_mx(plain_codes(c, bits, k), s, bits, k)


WIDE = [0, 1, 5, 9, 10, 11, 40, 63, 64, 100, 127, 127, 127, 150, 191, 192, 220, 245, 246, 247, 250, 254]


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("sizes_a,sizes_b", [(WIDE, WIDE), ([0, 3, 9, 10], [200, 240, 246, 247, 253]), ([247, 254], [0, 9, 20, 60]), ([0], [127, 130]),
                                             ([5, 127], [127, 249, 250])])
def test_scales_of_every_size(m, n, k, sizes_a, sizes_b, fa, fb):
    a, b = mixed(m, k, fa, m, sizes_a), mixed(n, k, fb, n + 1, sizes_b)
    ref, total = reference(a, b)
    fits = total < 2.0**127
    for out in (F32, BF16):
        got = spt.mx_matmul(a, b, out).to(F64)
        u = 0.0 if out == F32 else 2.0**-8
        tol = (k * 2.0**-23 + (2.0**-9 if out != F32 and fa == 8 else 0.0)) * total * (1 + u) + u * ref.abs() + k * 2.0**-126
        off = (got - ref).abs()
        assert (off[fits] <= tol[fits]).all(), (out, int((off[fits] > tol[fits]).sum()), float((off / tol)[fits].max()))
        beyond = (ref.abs() > 2.0**129) & (total < 1.5 * ref.abs())
        assert not torch.isfinite(got[beyond]).any()


@pytest.mark.parametrize("fb", [8, 4])
def test_blocks_without_a_number(fb):
    """A NaN block makes its row or column NaN beside far blocks too; rows without any get the bits that they get alone."""
    m, n, k = 50, 200, 700
    a, b = int_operand(m, k, 8, 3, spread=1), int_operand(n, k, fb, 4, spread=1)
    want = spt.mx_matmul(a, b, F32)
    x, y = scale_bytes(a)[:, :22].clone(), scale_bytes(b)[:, :22].clone()
    x[7, 3], x[9, 5], x[9, 6], y[11, 0] = 255, 2, 250, 251
    set_scales(a, x)
    set_scales(b, y)
    got = spt.mx_matmul(a, b, F32)
    assert torch.isnan(got[7]).all()
    rows = [i for i in range(m) if i not in (7, 9)]
    cols = [j for j in range(n) if j != 11]
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])
    ref, total = reference(a, b)
    # row 9's block at 2^123 passes fp32's end in every column: 32 products of magnitude 2 on average at 2^122 or more make about 2^128
    finite = total[9].nan_to_num(float("inf")) < 2.0**127
    assert ((got[9].to(F64) - ref[9]).abs() <= k * 2.0**-23 * total[9])[finite].all()
    beyond = (ref[9].abs() > 2.0**129) & (total[9] < 1.5 * ref[9].abs())
    assert not torch.isfinite(got[9])[beyond].any()


def test_real_rows_are_alike_beside_far_ones():
    """Gaussian rows: a far block in one row changes no bit of another."""
    for m, n, k in ((20, 300, 2000), (200, 500, 1500)):
        x, w = torch.randn((m, k), generator=gen(1), device="cuda"), torch.randn((n, k), generator=gen(2), device="cuda")
        b = spt.quantize_mx(w, 8)
        want = spt.mx_matmul(spt.quantize_mx(x, 8), b, F32)
        x[m // 2] *= 2.0**-120
        a = spt.quantize_mx(x, 8)
        got = spt.mx_matmul(a, b, F32)
        others = [i for i in range(m) if i != m // 2]
        assert torch.equal(got[others], want[others])
        ref, total = reference(a, b)
        assert ((got[m // 2].to(F64) - ref[m // 2]).abs() <= k * 2.0**-23 * total[m // 2] + k * 2.0**-126).all()
