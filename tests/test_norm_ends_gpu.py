"""GPU tests of the norm and its gradients whose results hang on single values: the ends of rows and of pieces, and every row of dweight.

Tolerances follow the kernels' own summation. A thread adds at most 8 max(4, ceil(n / 4096)) values of a row one after the other (four
pieces of eight, or n / 512 in two passes), and threads and waves add in pairs: ten levels. With D = that + 10 and v = 2^-24 a sum of
positive terms is off by D v, r = 1 / sqrt(mean + eps) by (D / 2 + 6) v (mean, eps, root and division as in test_norm_gpu.py), y by (D / 2 + 8) v
and the type's rounding; f = r^2 sum(g h) / n by (D + 16) v |f| + (D + 2) v r^2 sum|g h| / n.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402
from test_microscale_gpu import check_quantized, gen  # noqa: E402
from test_norm_gpu import TINY, V, plain, rand, u, weights  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
WIDTHS = [1, 3, 8, 9, 65, 100, 201, 512, 513, 1001, 1500, 2049, 4097, 8191, 8200, 9001, 12289, 16385, 20531, 32767, 32769, 39937, 40003, 70001]


def depth(n):
    return 8 * max(4, -(-n // 4096)) + 10


def places(n):
    """Columns at the ends of rows, pieces of eight, waves and workgroups' pieces, and some others."""
    cols = {0, 1, 7, 8, 63, 64, 511, 512, 1023, 1024, n // 2, n // 3, n - n % 8 - 1, n - n % 8, *(n - i for i in range(1, 18))}
    cols |= {c for p in (4096, 8192, 16384) for c in (p - 1, p)}
    return sorted(c for c in cols if 0 <= c < n)


def one_large(n, copies, dtype, seed, size):
    """Rows of normal values with one of `size` at each of the places in turn."""
    cols = places(n)
    x = rand((len(cols) * copies, n), F32, seed)
    x[torch.arange(x.shape[0]), torch.tensor(cols * copies)] = size
    return x.to(dtype)


def copies_of(n):
    """Some widths with many rows to a workgroup."""
    return 1 if n > 10000 else 130 if n in (100, 513, 1500, 4097) else 3


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_forward(n, dtype):
    """Squares of 4 n beside n - 1 of about 1: without the one value y would be 2.2 times as large."""
    x, w = one_large(n, copies_of(n), dtype, n, 2.0 * n**0.5), weights(n, F32, 2)
    r = rand(x.shape, dtype, 3, 0.1)
    y, h = spt.rms_norm(x, w, 1e-5, residual=r)
    for got, of in ((spt.rms_norm(x, w, 1e-5), x), (y, h)):
        ref, _ = plain(of, w, 1e-5)
        tol = (depth(n) / 2 + 8) * V * ref.abs() * (1 + u(dtype)) + u(dtype) * ref.abs() + TINY[dtype]
        assert ((got.to(F64) - ref).abs() <= tol).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", WIDTHS)
def test_microscaled(n, bits):
    """In fp32 the codes are those of the values that the norm itself returns."""
    x, w = one_large(n, copies_of(n), F32, n, 2.0 * n**0.5), weights(n, F32, 2)
    r = rand(x.shape, F32, 3, 0.1)
    check_quantized(spt.rms_norm_mx(x, w, 1e-5, bits=bits), spt.rms_norm(x, w, 1e-5))
    q, h = spt.rms_norm_mx(x, w, 1e-5, residual=r, bits=bits)
    y, s = spt.rms_norm(x, w, 1e-5, residual=r)
    assert torch.equal(h, s)
    check_quantized(q, y)


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gradient_of_rows(n, dtype):
    """sum(g h) hangs on one product: n against n - 1 of about 1 and either sign."""
    dy = one_large(n, copies_of(n), dtype, n, float(n) ** 0.5)
    cols = torch.tensor(places(n) * copies_of(n))
    h = rand(dy.shape, F32, 5)
    h[torch.arange(dy.shape[0]), cols] = float(n) ** 0.5
    h, w, dh = h.to(dtype), weights(n, F32, 6), rand(dy.shape, dtype, 7)
    d = depth(n)
    _, r = plain(h, None, 1e-5)
    g, hf = dy.to(F64) * w.to(F64), h.to(F64)
    f = r**2 * (g * hf).sum(dim=1, keepdim=True) / n
    ef = (d + 16) * V * f.abs() + (d + 2) * V * r**2 * (g * hf).abs().sum(dim=1, keepdim=True) / n
    parts = r * (g.abs() + hf.abs() * f.abs())
    for extra in (None, dh):
        dx, _ = spt.rms_norm_grad(dy, h, w, 1e-5, dh=extra)
        ref = r * (g - hf * f) + (0.0 if extra is None else extra.to(F64))
        tol = (d / 2 + 10) * V * parts + r * hf.abs() * ef + 2 * V * ref.abs()
        tol = tol * (1 + u(dtype)) + u(dtype) * ref.abs() + TINY[dtype]
        assert ((dx.to(F64) - ref).abs() <= tol).all()


ROWS = [(1, 77), (9001, 33), (5000, 200), (30000, 8), (3500, 1001), (2049, 1500), (20000, 1000), (9, 2560), (2048, 2560), (16384, 1024), (257, 3001),
        (300, 4096), (8191, 4096), (1300, 9001), (700, 17001), (530, 39936), (600, 39937), (100, 70001)]


@pytest.mark.parametrize("rows,n", ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_every_row_of_dweight(rows, n, dtype):
    """h of 1 and -1, so c = h r with the same r within 8 v of 1 in all rows, and whole dy of 1 to 3 without a zero: dweight is near a whole
    number that lacks no row. Sums of up to 30000 such terms of random sign, and of any part of them, stay below 2^12 (ten standard
    deviations of 2.2 sqrt(rows)), each of at most 400 additions (a workgroup's rows, planes by 64, 64 sums) rounds by 2^12 v: 0.1 in all."""
    g = gen(rows + n)
    h = (torch.randint(0, 2, (rows, n), generator=g, device="cuda") * 2 - 1).to(dtype)
    dy = ((torch.randint(0, 2, (rows, n), generator=g, device="cuda") * 2 - 1) * torch.randint(1, 4, (rows, n), generator=g, device="cuda")).to(dtype)
    w = weights(n, F32, 1)
    want = (dy.to(F64) * h.to(F64)).sum(dim=0)
    for extra in (None, dy):
        _, dw = spt.rms_norm_grad(dy, h, w, 0.0, dh=extra)
        assert (dw.to(F64) - want).abs().max() < 0.1
        assert torch.equal(dw.to(F64).round(), want)


@pytest.mark.parametrize("rows,n", [(2049, 1500), (257, 3001), (1300, 9001), (600, 20001), (5000, 100)])
def test_one_row_of_dweight(rows, n):
    """dy zero but for one row: dweight is that row's, wherever it lies among the workgroups."""
    h, w = rand((rows, n), BF16, 1), weights(n, F32, 2)
    _, r = plain(h, None, 1e-5)
    for row in sorted({0, 1, 3, 7, 8, 9, 15, 16, rows // 2, rows - 9, rows - 8, rows - 2, rows - 1}):
        dy = torch.zeros((rows, n), device="cuda", dtype=BF16)
        dy[row] = rand((n,), BF16, 3)
        _, dw = spt.rms_norm_grad(dy, h, w, 1e-5)
        ref = dy[row].to(F64) * h[row].to(F64) * r[row]
        assert ((dw.to(F64) - ref).abs() <= (depth(n) / 2 + 8) * V * ref.abs() + TINY[F32]).all()
