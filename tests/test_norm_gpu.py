"""GPU tests of the root-mean-square norm, its gradients and its microscaled form against 64 bits.

Tolerances count roundings, each off by at most half a step: u_t = eps_t / 2 of the value for type t, v = 2^-24 for
fp32. With n columns, the sum of squares adds positive terms: relative error at most n v + v, of which the root keeps
half; two more for mean and eps, one for the root and one for the division (each at most 2 v with fp32's own functions):
(n / 2 + 6) v for r. The kernel adds in a tree of depth far below n, so n is a bound, not a guess. y = h r w costs two products:
(n / 2 + 8) v |y|, then the type's rounding.
dx = r (g - h f) + dh: with S = sum |g h|, f = r^2 S' / n is off by (2 (n / 2 + 6) + 4) v |f| + (n + 2) v r^2 S / n.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402
from software_pipelined_tiled_amd import _lib  # noqa: E402
from test_microscale_gpu import check_quantized, codes_of, gen, scale_bytes, values  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
TINY = {F16: 2.0**-25, BF16: 2.0**-134, F32: 2.0**-150}
V = 2.0**-24
SIZES = [(1, 1), (1, 7), (3, 8), (2, 100), (65, 512), (5, 513), (7, 2048), (3, 2049), (130, 1000), (2, 4097), (9, 8192), (2, 8193),
         (3, 20000), (2, 32768), (3, 32769), (2, 70001), (1, 131072), (2500, 64)]


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def weights(n, dtype, seed):
    return None if dtype is None else (1.0 + 0.3 * torch.randn((n,), generator=gen(seed), device="cuda")).to(dtype)


def u(t):
    return torch.finfo(t).eps / 2


def summed(x, r):
    """h: exact in 64 bits, rounded once to the type."""
    return x if r is None else (x.to(F64) + r.to(F64)).to(x.dtype)


def plain(h, w, eps):
    h = h.to(F64)
    r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    return h * r * (1.0 if w is None else w.to(F64)), r


def check_y(y, h, w, eps):
    ref, _ = plain(h, w, eps)
    tol = (h.shape[1] / 2 + 8) * V * ref.abs() * (1 + u(y.dtype)) + u(y.dtype) * ref.abs() + TINY[y.dtype]
    off = (y.to(F64) - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("dtype,wtype", [(F16, F16), (BF16, F32), (F32, F32), (BF16, None), (F32, BF16), (F16, F32)])
def test_forward(rows, n, dtype, wtype):
    x, r, w = rand((rows, n), dtype, rows + n), rand((rows, n), dtype, 1), weights(n, wtype, 2)
    y = spt.rms_norm(x, w, 1e-5)
    assert y.dtype == dtype
    check_y(y, x, w, 1e-5)
    y, h = spt.rms_norm(x, w, 1e-5, residual=r)
    # fp32 adds once and rounds again to 16 bits: where that lands on a middle the two roundings may differ from one by a step
    want = summed(x, r)
    assert torch.equal(h, want) or (dtype != F32 and ((h.float() - want.float()).abs() <= 2 * u(dtype) * want.float().abs() * 1.01).all()
                                    and (h != want).float().mean() < 1e-3)
    check_y(y, h, w, 1e-5)
    assert torch.equal(y, spt.rms_norm(h, w, 1e-5))  # the norm of what is returned


def grad_reference(dy, h, w, eps, dh):
    """dx, dw and their tolerances before the types' rounding (the file's head)."""
    n, rows = h.shape[1], h.shape[0]
    _, r = plain(h, None, eps)
    hf, dyf, wf = h.to(F64), dy.to(F64), 1.0 if w is None else w.to(F64)
    g = dyf * wf
    s, total = (g * hf).sum(dim=1, keepdim=True), (g * hf).abs().sum(dim=1, keepdim=True)
    f = r**2 * s / n
    dx = r * (g - hf * f) + (0.0 if dh is None else dh.to(F64))
    er = (n / 2 + 6) * V
    ef = (2 * er + 4 * V) * f.abs() + (n + 2) * V * r**2 * total / n
    parts = r * (g.abs() + hf.abs() * f.abs())
    tol_dx = (er + 4 * V) * parts + r * hf.abs() * ef + 2 * V * dx.abs()
    dw = (dyf * hf * r).sum(dim=0)
    tol_dw = (er + (rows + 3) * V) * (dyf * hf * r).abs().sum(dim=0)
    return dx, tol_dx, dw, tol_dw


def within(got, ref, tol):
    t = got.dtype
    tol = tol * (1 + u(t)) + u(t) * ref.abs() + TINY[t]
    off = (got.to(F64) - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("dtype,wtype", [(F16, F16), (BF16, F32), (F32, F32), (BF16, BF16), (F32, None)])
def test_gradients(rows, n, dtype, wtype):
    h, dy, dh = rand((rows, n), dtype, 3), rand((rows, n), dtype, 4), rand((rows, n), dtype, 5)
    w = weights(n, wtype, 6)
    for d in (None, dh):
        dx, dw = spt.rms_norm_grad(dy, h, w, 1e-5, dh=d)
        rx, tx, rw, tw = grad_reference(dy, h, w, 1e-5, d)
        within(dx, rx, tx)
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == wtype
            within(dw, rw, tw)


@pytest.mark.parametrize("rows,n", [(9001, 33), (3500, 1001), (2049, 1500), (20000, 1000), (9, 2560), (257, 3001), (1300, 9001), (700, 17001), (530, 39936), (600, 39937)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_rows(rows, n, dtype):
    """Several rows to a workgroup: what is kept from row to row, and the sums over rows, of rows of every length."""
    h, dy, dh, w = rand((rows, n), dtype, 3), rand((rows, n), dtype, 4), rand((rows, n), dtype, 5), weights(n, F32, 6)
    dx, dw = spt.rms_norm_grad(dy, h, w, 1e-5, dh=dh)
    rx, tx, rw, tw = grad_reference(dy, h, w, 1e-5, dh)
    within(dx, rx, tx)
    within(dw, rw, tw)
    del dx, rx, tx
    y, s = spt.rms_norm(dy, w, 1e-5, residual=dh)
    check_y(y, s, w, 1e-5)
    # each row's result is its own: rows in another order and number give the same bits
    pick = torch.arange(rows - 1, -1, -3, device="cuda")
    assert torch.equal(spt.rms_norm(dy[pick], w, 1e-5, residual=dh[pick])[0], y[pick])
    q = spt.rms_norm_mx(s, w, 1e-5, bits=8)
    few = spt.rms_norm_mx(s[pick], w, 1e-5, bits=8)
    assert torch.equal(spt.dequantize_mx(q, dtype)[pick], spt.dequantize_mx(few, dtype))


def test_gradients_against_differences():
    """Central differences in 64 bits of the definition against the kernel's fp32 gradients: with steps of 2^-10 the cubic term
    of a function of unit scale is below 2^-18."""
    rows, n, eps = 3, 40, 1e-3
    x, r, w = rand((rows, n), F32, 1), rand((rows, n), F32, 2), weights(n, F32, 3)
    dy, dh = rand((rows, n), F32, 4), rand((rows, n), F32, 5)

    def loss(xd, rd, wd):
        h = xd + rd
        return (h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps) * wd * dy.double()).sum() + (h * dh.double()).sum()

    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = spt.rms_norm(leaves[0], leaves[1], eps, residual=leaves[2])
    grads = torch.autograd.grad((y, h), leaves, (dy, dh))
    step = 2.0**-10
    for which, got in zip((0, 2, 1), grads):
        args = [x.double(), r.double(), w.double()]
        flat = args[which].reshape(-1)
        for i in range(0, flat.numel(), 7):
            at = flat[i].item()
            flat[i] = at + step
            hi = loss(*args)
            flat[i] = at - step
            lo = loss(*args)
            flat[i] = at
            assert abs((hi - lo).item() / (2 * step) - got.reshape(-1)[i].item()) < 2e-4


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("extra,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_strides(dtype, extra, offset):
    rows, n = 35, 777

    def strided(t, fill=float("nan")):
        buf = torch.full((rows * (n + extra) + offset,), fill, dtype=dtype, device="cuda")
        v = buf[offset:].view(rows, n + extra)
        v[:, :n] = t
        return v

    x, r, dy, dh = (rand((rows, n), dtype, i) for i in range(4))
    w = weights(n + 1, dtype, 9)[1:]
    y, h = spt.rms_norm(x, w, residual=r)
    sy, sh = strided(torch.zeros_like(x), 7.0), strided(torch.zeros_like(x), 7.0)
    spt.rms_norm(strided(x)[:, :n], w, residual=strided(r)[:, :n], out=sy[:, :n], residual_out=sh[:, :n])
    assert torch.equal(sy[:, :n], y) and torch.equal(sh[:, :n], h) and (sy[:, n:] == 7.0).all() and (sh[:, n:] == 7.0).all()
    dx, dw = spt.rms_norm_grad(dy, h, w, dh=dh)
    ex, ew = spt.rms_norm_grad(strided(dy)[:, :n], strided(h)[:, :n], w, dh=strided(dh)[:, :n])
    assert torch.equal(dx, ex) and torch.equal(dw, ew)
    for bits in (4, 8):
        q = spt.rms_norm_mx(x, w, bits=bits)
        p = spt.rms_norm_mx(strided(x)[:, :n], w, bits=bits)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)


@pytest.mark.parametrize("n", [1, 7, 100, 201, 4096, 8191, 20531, 40000, 40003])
def test_in_place(n):
    """The residual's stream kept in one tensor, as a decoding loop does."""
    x, r, w = rand((5, n), BF16, 1), rand((5, n), BF16, 2), weights(n, BF16, 3)
    y, h = spt.rms_norm(x, w, residual=r)
    keep = r.clone()
    y1, h1 = spt.rms_norm(x, w, residual=keep, residual_out=keep)
    assert h1.data_ptr() == keep.data_ptr() and torch.equal(keep, h) and torch.equal(y1, y)
    keep = x.clone()
    y1, _ = spt.rms_norm(keep, w, residual=r, residual_out=keep)
    assert torch.equal(keep, h) and torch.equal(y1, y)
    keep = x.clone()
    assert torch.equal(spt.rms_norm(keep, w, out=keep), spt.rms_norm(x, w))
    a, b, keep = x.clone(), None, r.clone()
    spt.rms_norm(a, w, residual=keep, out=a, residual_out=keep)
    assert torch.equal(a, y) and torch.equal(keep, h)
    keep = r.clone()
    q, h1 = spt.rms_norm_mx(x, w, residual=keep, residual_out=keep)
    p, _ = spt.rms_norm_mx(x, w, residual=r)
    assert torch.equal(keep, h) and torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)


@pytest.mark.parametrize("n", [3, 201, 1001, 9001, 20531, 40003])
@pytest.mark.parametrize("over", ["dy", "dh"])
def test_gradient_over_its_operand(n, over):
    """dx in dy's or dh's own memory, as the C interface allows."""
    rows = 300
    h, w = rand((rows, n), BF16, 1), weights(n, F32, 2)
    t = {"dy": rand((rows, n), BF16, 3), "dh": rand((rows, n), BF16, 4)}
    want_dx, want_dw = spt.rms_norm_grad(t["dy"], h, w, 1e-6, dh=t["dh"])
    dw = torch.empty_like(w)
    p = _lib.NormRmsGrad(rows, n, spt.GEMM_BF16, spt.GEMM_F32, 1e-6, n, n, n, n)
    size = _lib.norm_rms_grad_workspace_bytes(p, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert spt.lib().norm_rms_grad_run(p, t["dy"].data_ptr(), h.data_ptr(), w.data_ptr(), t["dh"].data_ptr(), t[over].data_ptr(),
                                       dw.data_ptr(), ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(t[over], want_dx) and torch.equal(dw, want_dw)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 33), (64, 128), (65, 100), (130, 1000), (600, 512), (2, 4097), (70, 8192), (3, 33000), (1, 70000)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_mx(rows, n, dtype, bits):
    """The codes are those of y to within y's own error: the quantised values lie between what y's two bounds quantise to."""
    x, r, w = rand((rows, n), dtype, rows + n), rand((rows, n), dtype, 1), weights(n, F32, 2)
    q, h = spt.rms_norm_mx(x, w, 1e-5, residual=r, bits=bits)
    y, h2 = spt.rms_norm(x, w, 1e-5, residual=r)
    assert torch.equal(h, h2) and q.shape == (rows, n) and q.bits == bits
    check_near(q, h, w, 1e-5)
    check_near(spt.rms_norm_mx(x, w, 1e-5, bits=bits), x, w, 1e-5)


def check_near(q, h, w, eps):
    """Every scale and value is what some y within the tolerance gives: the scale is that of the block's largest, which may
    sit at a power of two; given the scale, rounding is monotonic."""
    ref, _ = plain(h, w, eps)
    rows, n = ref.shape
    off = (n / 2 + 8) * V * ref.abs() + TINY[F32]
    s = scale_bytes(q).long()
    full = torch.zeros((rows, s.shape[1] * 32), dtype=F64, device="cuda")
    lo, hi = full.clone(), full.clone()
    lo[:, :n], hi[:, :n] = (ref.abs() - off).clamp(min=0.0), ref.abs() + off
    emax = 2 if q.bits == 4 else 8

    def scale(v):
        top = v.view(rows, -1, 32).amax(dim=2)
        _, e = torch.frexp(top)
        return torch.where(top > 0, torch.clamp(e.long() - 1 - emax + 127, min=0), 0)

    assert ((s >= scale(lo)) & (s <= scale(hi))).all()
    from test_microscale_gpu import levels, power
    table = levels(q.bits)[: 8 if q.bits == 4 else 127]
    mid = (table[1:] + table[:-1]) / 2
    unit = power(127 - s).repeat_interleave(32, dim=1)
    code = codes_of(q) % (8 if q.bits == 4 else 128)
    assert ((code >= torch.bucketize(lo * unit, mid)) & (code <= torch.bucketize(hi * unit, mid, right=True))).all()
    sign = codes_of(q)[:, :n] >= (8 if q.bits == 4 else 128)
    assert (sign == torch.signbit(ref))[ref != 0].all()
    assert not codes_of(q)[:, n:].any()
    if rows % 64:
        assert not q.scales[-1, :, rows % 64:].any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,n", [(13001, 1001), (12290, 4096), (2603, 9001), (1030, 8192), (2570, 17001), (5001, 600)])
def test_mx_of_many_rows(rows, n, bits):
    """Codes and scales of workgroups with several rows, from any row of four on, are those of few rows at a time, the zeros behind the
    last row too."""
    x, w = rand((rows, n), BF16, 1), weights(n, BF16, 2)
    q = spt.rms_norm_mx(x, w, bits=bits)
    for at in range(0, rows, 64 * 41):
        part = spt.rms_norm_mx(x[at: at + 128], w, bits=bits)
        blocks = part.scales.shape[0]
        assert torch.equal(q.codes[at: at + 128], part.codes)
        assert torch.equal(q.scales[at // 64: at // 64 + blocks], part.scales)
    at = rows // 64 * 64 - 64
    part = spt.rms_norm_mx(x[at:], w, bits=bits)
    assert torch.equal(q.scales[at // 64:], part.scales) and (part.scales[-1, :, (rows - 1) % 64 + 1:] == 0).all()


def test_mx_feeds_the_product():
    """A layer: norm in 8 bits, product with a 4-bit weight; against the norm in fp32 quantised by itself."""
    x, r, w = rand((50, 1000), F32, 1), rand((50, 1000), F32, 2), weights(1000, F32, 3)
    b = spt.quantize_mx(rand((300, 1000), F32, 4), 4)
    q, h = spt.rms_norm_mx(x, w, residual=r)
    y, _ = spt.rms_norm(x, w, residual=r)
    check_quantized(q, y)  # y is fp32 here: what was quantised
    assert torch.equal(spt.mx_matmul(q, b, BF16), spt.mx_linear(y, b, out_dtype=BF16))
    ref = values(q) @ values(b).t()
    assert ((spt.mx_matmul(q, b, F32).double() - ref).norm() / ref.norm()) < 1e-6


def test_not_finite_rows():
    """A row with an infinity or a NaN is NaN (the infinity's own place too: inf / inf), and no other row is."""
    x = rand((6, 300), F32, 1)
    x[1, 5], x[3, 7], x[4] = float("nan"), float("inf"), 0.0
    y = spt.rms_norm(x, None, 1e-5)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 7]) and torch.isfinite(y[[0, 2, 4, 5]]).all() and not y[4].any()
    q = spt.rms_norm_mx(x, None, 1e-5)
    s = scale_bytes(q)
    assert (s[1, :10] == 255).all() and (s[[0, 2, 4, 5]] < 255).all() and not s[4].any() and not s[1, 10:].any()


def test_empty():
    w = torch.ones(10, device="cuda")
    x = torch.empty((0, 10), device="cuda")
    assert spt.rms_norm(x, w).shape == (0, 10)
    dx, dw = spt.rms_norm_grad(x, x, w)
    assert dx.shape == (0, 10) and dw.shape == (10,) and not dw.any()
    e = torch.empty((4, 0), device="cuda")
    assert spt.rms_norm(e).shape == (4, 0)
    dx, dw = spt.rms_norm_grad(e, e, torch.empty(0, device="cuda"))
    assert dx.shape == (4, 0) and dw.shape == (0,)
    assert spt.rms_norm_mx(x, w).shape == (0, 10) and spt.rms_norm_mx(e).shape == (4, 0)


def test_autograd():
    rows, n = 33, 500
    x, r = rand((rows, n), BF16, 1).requires_grad_(), rand((rows, n), BF16, 2).requires_grad_()
    w = weights(n, F32, 3).requires_grad_()
    dy, dh = rand((rows, n), BF16, 4), rand((rows, n), BF16, 5)
    with torch.no_grad():
        h = spt.rms_norm(x, w, residual=r)[1]
        want = spt.rms_norm_grad(dy, h, w, dh=dh)
        alone = spt.rms_norm_grad(dy, h, w)
        first = spt.rms_norm_grad(dy, x, w)
    y, hg = spt.rms_norm(x, w, residual=r)
    gx, gr, gw = torch.autograd.grad((y, hg), (x, r, w), (dy, dh))
    assert torch.equal(gx, want[0]) and torch.equal(gr, want[0]) and torch.equal(gw, want[1])
    y, hg = spt.rms_norm(x, w, residual=r)
    gx, gw = torch.autograd.grad(y, (x, w), dy)  # h unused
    assert torch.equal(gx, alone[0]) and torch.equal(gw, alone[1])
    y, hg = spt.rms_norm(x, w, residual=r)
    gx, gw = torch.autograd.grad(hg, (x, w), dh, allow_unused=True)  # y unused
    assert torch.equal(gx, dh) and gw is None
    gx, gw = torch.autograd.grad(spt.rms_norm(x, w), (x, w), dy)
    assert torch.equal(gx, first[0]) and torch.equal(gw, first[1])
    # one of the inputs alone, and one tensor as both
    assert torch.equal(torch.autograd.grad(spt.rms_norm(x.detach(), w), w, dy)[0], first[1])
    assert torch.equal(torch.autograd.grad(spt.rms_norm(x, w.detach()), x, dy)[0], first[0])
    y, _ = spt.rms_norm(x, w, residual=x)
    with torch.no_grad():
        both = spt.rms_norm_grad(dy, (x.float() * 2).to(BF16), w)[0]
    assert torch.equal(torch.autograd.grad(y, x, dy)[0], both + both)
    # a broadcast and a transposed gradient
    y = spt.rms_norm(x, w)
    a = torch.autograd.grad(y, x, torch.ones((1, 1), device="cuda", dtype=BF16).expand(rows, n))[0]
    with torch.no_grad():
        assert torch.equal(a, spt.rms_norm_grad(torch.ones_like(x), x, w)[0])
    y = spt.rms_norm(x, w)
    assert torch.equal(torch.autograd.grad(y, x, dy.t().contiguous().t())[0], first[0])


@pytest.mark.parametrize("rows,n", [(300, 1000), (600, 20001), (3, 60)])
def test_captured_step(rows, n):
    """Forward and both gradients by plain calls in one graph, replayed on new values."""
    x, r, w = rand((rows, n), BF16, 1), rand((rows, n), BF16, 2), weights(n, F32, 3)
    dy, dh = rand((rows, n), BF16, 4), rand((rows, n), BF16, 5)

    def step():
        y, h = spt.rms_norm(x, w, residual=r)
        return (y, h, *spt.rms_norm_grad(dy, h, w, dh=dh))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for turn in range(4):
        x.copy_(rand((rows, n), BF16, 20 + turn))
        dy.copy_(rand((rows, n), BF16, 40 + turn))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_same_bits_every_run():
    h, dy, w = rand((5000, 900), BF16, 1), rand((5000, 900), BF16, 2), weights(900, F32, 3)
    first = spt.rms_norm_grad(dy, h, w)
    for _ in range(5):
        again = spt.rms_norm_grad(dy, h, w)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
