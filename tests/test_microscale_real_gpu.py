"""GPU tests of products of real values through every kernel, whole and in parts, against 64 bits.

Element by element: an fp32 sum of k terms of total magnitude T is off by at most k 2^-23 T, whatever its order; with operands of 8 bits and a
16-bit result the matrix instructions cut what lies 13 bits below the largest of up to 16 products: 2^-9 T more; then the type's rounding.

Over all results, which such bounds do not see: on Gaussian data the sums are off by e of the results' norm, 1.5e-5 for 8 x 8, 5e-6 for
8 x 4 and by what fp32 sums lose, here 1e-6, for 4 x 4 and fp32 results. Where an error d moves a result over a middle between two neighbours s
apart, which has the probability |d| / s, the rounded result differs by s from the rounded exact one: the expected sum of squares is
sum(s |d|), with s <= 2 u |exact| at most 2 u |exact|_2 |d|_2, so the relative norm is sqrt(2 u e). 1.5 times that for chance (the
shapes have 2000 results or more), and e itself where the type is fp32.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402
from microscale_cases import FORMATS, REAL  # noqa: E402
from test_microscale_gpu import TINY, gen, plain_codes, reference  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
SUM_ERROR = {(8, 8): 1.5e-5, (8, 4): 5e-6, (4, 4): 1e-6}
FP32_ERROR = 1e-6


def normal(shape, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda")


def any_codes(rows, k, bits, seed):
    """Every number of the format (no NaN), scales of 2^-3 .. 2^2."""
    g = gen(seed)
    sign = torch.randint(0, 2, (rows, k), generator=g, device="cuda") * (8 if bits == 4 else 128)
    codes = torch.randint(0, 8 if bits == 4 else 127, (rows, k), generator=g, device="cuda") + sign
    scales = torch.randint(124, 130, (rows, -(-k // 32)), generator=g, device="cuda").to(torch.uint8)
    return spt.pack_mx(plain_codes(codes, bits, k), scales, bits, k)


def within(got, ref, total, k, fa):
    u = torch.finfo(got.dtype).eps / 2
    err = (k * 2.0**-23 + (2.0**-9 if fa == 8 and got.dtype != F32 else 0.0)) * total
    fits = ref.abs() + err < torch.finfo(got.dtype).max * (1 - u)
    tol = err * (1 + u) + u * ref.abs() + TINY[got.dtype]
    off = (got.to(F64) - ref).abs()
    # sums of 12046 products of e4m3's whole range have magnitudes of 10^7 in total, beyond fp16 in every element
    assert fits.any() or (got.dtype == F16 and total.min() > 2.0**16)
    assert (off <= tol)[fits].all(), (int((off > tol)[fits].sum()), (off / tol)[fits].amax(dim=0))


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", REAL)
def test_every_number_of_the_format(m, n, k, fa, fb):
    a, b = any_codes(m, k, fa, m + k), any_codes(n, k, fb, n + k + 1)
    ref, total = reference(a, b)
    for out in (F32, BF16, F16):
        got = spt.mx_matmul(a, b, out)
        within(got, ref, total, k, fa)
        if out == F32:
            assert ((got.to(F64) - ref).norm() / ref.norm()).item() < FP32_ERROR


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", REAL)
def test_gaussian_rows(m, n, k, fa, fb):
    a, b = spt.quantize_mx(normal((m, k), m), fa), spt.quantize_mx(normal((n, k), n + 1), fb)
    ref, total = reference(a, b)
    for out in (F32, BF16, F16):
        got = spt.mx_matmul(a, b, out)
        within(got, ref, total, k, fa)
        off = ((got.to(F64) - ref.to(F32).to(out).to(F64)).norm() / ref.norm()).item()
        if out == F32:
            assert off < FP32_ERROR
        else:
            u = torch.finfo(out).eps / 2
            assert off < 1.5 * (2 * u * SUM_ERROR[fa, fb]) ** 0.5, off


# SUM_ERROR where one column of A in 200 is twenty times the others, and anywhere: with independent signs the squares of a result's terms add
# up, and in each group of 16 the 15 others lose less than 2^-13 of the largest, whose square is among them: sqrt(15) 2^-13 = 4.8e-4. Products
# of two 4-bit values lose nothing.
LARGE_COLUMNS = {(8, 8): 15**0.5 * 2.0**-13, (8, 4): 15**0.5 * 2.0**-13, (4, 4): 1e-6}


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("m,n,k", [(m, n, -(-k // 64) * 64) for m, n, k in REAL])
def test_sums_that_cancel(m, n, k, fa, fb, large):
    """Rows [x, x'] and [w, -w'], x' and w' the values of x and w in another order inside their blocks, and the blocks in another order: the
    exact result is zero, and what comes out is the two halves' error, sqrt(2) e of a half's norm if they know nothing of each other."""
    x, w = normal((m, k // 2), m), normal((n, k // 2), n + 1)
    if large:
        x[:, ::200] *= 20.0
    inside = torch.rand((k // 64, 32), generator=torch.Generator().manual_seed(1)).argsort(dim=1).cuda()
    order = torch.randperm(k // 64, generator=torch.Generator().manual_seed(2)).cuda()

    def moved(t):
        t = t.view(t.shape[0], -1, 32)
        return t.gather(2, inside.expand(t.shape[0], -1, -1))[:, order].reshape(t.shape[0], -1)

    a, b = spt.quantize_mx(torch.cat([x, moved(x)], dim=1), fa), spt.quantize_mx(torch.cat([w, -moved(w)], dim=1), fb)
    half, _ = reference(spt.quantize_mx(x, fa), spt.quantize_mx(w, fb))
    ref, total = reference(a, b)
    for out in (F32, BF16, F16):
        got = spt.mx_matmul(a, b, out)
        within(got, ref, total, k, fa)
        e = FP32_ERROR if out == F32 else (LARGE_COLUMNS if large else SUM_ERROR)[fa, fb]
        assert (got.to(F64).norm() / half.norm()).item() < 2.0**0.5 * e
