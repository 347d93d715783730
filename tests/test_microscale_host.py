"""Microscaled tensors, their products and the norm on a host without a GPU: the header's symbols are exported and bound, sizes
of layouts and workspaces, and every refusal the C ABI and the torch face make before any device work."""
import ctypes
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

import software_pipelined_tiled_amd as spt
from software_pipelined_tiled_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = _lib.GEMM_OK, _lib.GEMM_ERR_INVALID, _lib.GEMM_ERR_UNSUPPORTED
F16, BF16, F32 = spt.GEMM_F16, spt.GEMM_BF16, spt.GEMM_F32
A, ODD = 0x1000, 0x1008  # addresses that no refused call reads: on 16 bytes, and off them
ROWS, K = 2**31 - 64, 2**22


def test_library_exports_every_header_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "microscale.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"gemm_status_t\s+(\w+)\s*\(", text)))
    assert names == sorted(spt.MX_EXPORTS)
    for n in names:
        assert hasattr(spt.lib(), n), n


@pytest.mark.parametrize("struct,name", [(_lib.GemmMx, "gemm_mx_t"), (_lib.NormRms, "norm_rms_t"), (_lib.NormRmsGrad, "norm_rms_grad_t")])
def test_structs_match_the_header(struct, name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "microscale.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
    kinds = {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "gemm_dtype_t": ctypes.c_int, "float": ctypes.c_float}
    want = [(field.strip(), kinds[line.split()[0]]) for line in body.split(";") if line.strip()
            for field in line.strip().split(None, 1)[1].split(",")]
    assert struct._fields_ == want


# ------------------------------------------------------------------------------- microscaled tensors

def sizes(rows, k, bits):
    c, s = ctypes.c_int64(-7), ctypes.c_int64(-7)
    return spt.lib().mx_bytes(rows, k, bits, ctypes.byref(c), ctypes.byref(s)), c.value, s.value


@pytest.mark.parametrize("rows,k", [(0, 0), (0, 5), (5, 0), (1, 1), (64, 128), (65, 129), (1000, 4100), (ROWS, K)])
@pytest.mark.parametrize("bits", [4, 8])
def test_bytes(rows, k, bits):
    blocks = -(-k // 128) * 4
    assert sizes(rows, k, bits) == (OK, rows * blocks * 4 * bits, -(-rows // 64) * 64 * blocks)


@pytest.mark.parametrize("rows,k,bits,status", [(-1, 5, 8, INVALID), (5, -1, 8, INVALID), (5, 5, 6, INVALID), (5, 5, 0, INVALID),
                                                (ROWS + 1, 5, 8, UNSUPPORTED), (5, K + 1, 4, UNSUPPORTED)])
def test_size_refusals(rows, k, bits, status):
    L, n = spt.lib(), ctypes.byref(ctypes.c_int64())
    assert sizes(rows, k, bits)[0] == status
    assert L.mx_quantize(A, BF16, rows, k, K + 8, bits, A, A, None) == status
    assert L.mx_dequantize(A, A, bits, rows, k, A, F32, K + 8, None) == status
    assert L.mx_pack(A, K + 8, A, K + 8, bits, rows, k, A, A, None) == status
    for m, nn in ((rows, 4), (4, rows)):
        p = _lib.GemmMx(m, nn, k, bits, bits, BF16, max(nn, 4))
        assert L.gemm_mx_workspace_bytes(ctypes.byref(p), n) in (status, INVALID if nn < 0 else status)
        assert L.gemm_mx_run(ctypes.byref(p), A, A, A, A, A, A, 1 << 62, None) in (status, INVALID if nn < 0 else status)
    assert L.mx_bytes(4, 4, 8, None, n) == INVALID and L.mx_bytes(4, 4, 8, n, None) == INVALID


@pytest.mark.parametrize("args,status", [
    ((A, 7, 4, 40, 40, 8, A, A), INVALID), ((A, BF16, 4, 40, 39, 8, A, A), INVALID), ((None, BF16, 4, 40, 40, 8, A, A), INVALID),
    ((A, BF16, 4, 40, 40, 8, None, A), INVALID), ((A, BF16, 4, 40, 40, 8, A, None), INVALID), ((A, BF16, 4, 40, 40, 8, ODD, A), INVALID),
    ((A, BF16, 4, 40, 40, 4, A, ODD), INVALID), ((None, F32, 0, 40, 40, 4, None, None), OK), ((None, F16, 4, 0, 0, 8, None, None), OK)])
def test_quantize_refusals(args, status):
    assert spt.lib().mx_quantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A, A, 8, 4, 40, A, 3, 40), INVALID), ((A, A, 8, 4, 40, A, F32, 39), INVALID), ((None, A, 8, 4, 40, A, F32, 40), INVALID),
    ((A, None, 8, 4, 40, A, F32, 40), INVALID), ((A, A, 8, 4, 40, None, F32, 40), INVALID), ((ODD, A, 8, 4, 40, A, F32, 40), INVALID),
    ((A, ODD, 4, 4, 40, A, F32, 40), INVALID), ((None, None, 4, 0, 40, None, F16, 40), OK), ((None, None, 8, 4, 0, None, F16, 0), OK)])
def test_dequantize_refusals(args, status):
    assert spt.lib().mx_dequantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A, 39, A, 2, 8, 4, 40, A, A), INVALID), ((A, 20, A, 1, 4, 4, 41, A, A), INVALID), ((A, 40, A, 1, 8, 4, 40, A, A), INVALID),
    ((None, 40, A, 2, 8, 4, 40, A, A), INVALID), ((A, 40, None, 2, 8, 4, 40, A, A), INVALID), ((A, 40, A, 2, 8, 4, 40, None, A), INVALID),
    ((A, 40, A, 2, 8, 4, 40, A, None), INVALID), ((A, 40, A, 2, 8, 4, 40, ODD, A), INVALID), ((A, 40, A, 2, 8, 4, 40, A, ODD), INVALID),
    ((None, 40, None, 2, 8, 0, 40, None, None), OK), ((None, 0, None, 0, 4, 4, 0, None, None), OK)])
def test_pack_refusals(args, status):
    assert spt.lib().mx_pack(*args, None) == status


# ------------------------------------------------------------------------------------------ products

def product(change):
    c = dict(m=40, n=48, k=200, a_bits=8, b_bits=8, out_dtype=BF16, ldc=48, a=A, sa=A, b=A, sb=A, c=A, ws=A, bytes=1 << 40)
    c.update(change)
    return _lib.GemmMx(*(c[f] for f, _ in _lib.GemmMx._fields_)), [c[f] for f in ("a", "sa", "b", "sb", "c", "ws", "bytes")]


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-1), INVALID), (dict(a_bits=6), INVALID), (dict(b_bits=16), INVALID),
    (dict(out_dtype=4), INVALID), (dict(ldc=47), INVALID), (dict(a_bits=4), UNSUPPORTED), (dict(a_bits=4, b_bits=4), None),
    (dict(b_bits=4), None), (dict(ldc=2**20), UNSUPPORTED), (dict(ldc=2**20 - 1), None), (dict(k=K + 1), UNSUPPORTED), (dict(k=K), None),
    (dict(m=ROWS + 1), UNSUPPORTED), (dict(n=2**20 - 1, ldc=2**20 - 1), None), (dict(m=2**29, n=64), None),
    (dict(m=2**29 + 1, n=64, ldc=64), UNSUPPORTED), (dict(m=2**29, n=65, ldc=65), UNSUPPORTED),
    (dict(m=2**15, n=2**20 - 1, ldc=2**20 - 1), None), (dict(m=2**15 + 1, n=2**20 - 1, ldc=2**20 - 1), UNSUPPORTED)])
def test_product_refusals(change, status):
    """status None: taken, by the size of its workspace."""
    change = dict(dict(ldc=max(48, change.get("n", 48))), **change)
    p, args = product(change)
    size = ctypes.c_int64(-7)
    got = spt.lib().gemm_mx_workspace_bytes(ctypes.byref(p), ctypes.byref(size))
    assert got == (OK if status is None else status)
    if status is None:
        assert 0 <= size.value <= 16 * p.m * p.n * 4
    else:
        assert spt.lib().gemm_mx_run(ctypes.byref(p), *args, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID), (dict(c=None), INVALID),
    (dict(a=ODD), INVALID), (dict(sa=ODD), INVALID), (dict(b=ODD), INVALID), (dict(sb=ODD), INVALID),
    (dict(m=0, a=None, sa=None, c=None), OK), (dict(n=0, b=None, sb=None, c=None), OK), (dict(k=0, c=None), INVALID)])
def test_product_pointers(change, status):
    p, args = product(change)
    assert spt.lib().gemm_mx_run(ctypes.byref(p), *args, None) == status
    assert spt.lib().gemm_mx_run(None, *args, None) == INVALID
    assert spt.lib().gemm_mx_workspace_bytes(ctypes.byref(p), None) == INVALID


@pytest.mark.parametrize("bits", [(8, 8), (8, 4), (4, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_product_workspace(bits, dtype):
    """A long sum of few tiles is cut, and its planes have to be there."""
    p, args = product(dict(m=100, n=33, k=40000, a_bits=bits[0], b_bits=bits[1], out_dtype=dtype))
    need = _lib.gemm_mx_workspace_bytes(p)
    assert need > 0 and need % (100 * 33 * 4) == 0
    for ws, size in ((None, need), (ODD, need), (A, need - 1), (A, 0)):
        assert spt.lib().gemm_mx_run(ctypes.byref(p), *args[:5], ws, size, None) == INVALID
    p, _ = product(dict(m=100, n=33, k=200, a_bits=bits[0], b_bits=bits[1], out_dtype=dtype))
    assert _lib.gemm_mx_workspace_bytes(p) == 0


# ---------------------------------------------------------------------------------------------- norm

def norm(change):
    c = dict(rows=4, n=40, dtype=BF16, weight_dtype=F32, eps=1e-6, ldx=40, ldr=40, ldh=40, ldy=40, x=A, r=A, w=A, h=A, y=A, s=A)
    c.update(change)
    return _lib.NormRms(*(c[f] for f, _ in _lib.NormRms._fields_)), c


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(dtype=3), INVALID), (dict(weight_dtype=-1), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(ldx=39), INVALID), (dict(ldr=39), INVALID),
    (dict(ldh=39), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(h=None), INVALID), (dict(rows=ROWS + 1), UNSUPPORTED),
    (dict(n=2**24 + 1, ldx=2**25, ldr=2**25, ldh=2**25, ldy=2**25), UNSUPPORTED), (dict(rows=0, x=None, y=None, h=None), OK),
    (dict(n=0, x=None, y=None, h=None), OK)])
def test_norm_refusals(change, status):
    p, c = norm(change)
    assert spt.lib().norm_rms_run(ctypes.byref(p), c["x"], c["r"], c["w"], c["h"], c["y"], None) == status
    for bits in (4, 8):
        assert spt.lib().norm_rms_mx_run(ctypes.byref(p), bits, c["x"], c["r"], c["w"], c["h"], c["y"], c["s"], None) == status


def test_norm_refusals_of_one_result():
    p, c = norm(dict(ldy=39))
    assert spt.lib().norm_rms_run(ctypes.byref(p), A, A, A, A, A, None) == INVALID
    p, c = norm({})
    for bits, y, s in ((5, A, A), (0, A, A), (8, ODD, A), (4, A, ODD), (4, A, None)):
        assert spt.lib().norm_rms_mx_run(ctypes.byref(p), bits, A, A, A, A, y, s, None) == INVALID
    p, c = norm(dict(n=K + 1, ldx=K + 1, ldr=K + 1, ldh=K + 1))
    assert spt.lib().norm_rms_mx_run(ctypes.byref(p), 8, A, A, A, A, A, A, None) == UNSUPPORTED
    assert spt.lib().norm_rms_run(None, A, A, A, A, A, None) == INVALID
    assert spt.lib().norm_rms_mx_run(None, 8, A, A, A, A, A, A, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(dtype=3), INVALID), (dict(weight_dtype=3), INVALID), (dict(eps=-1.0), INVALID),
    (dict(lddy=39), INVALID), (dict(ldh=39), INVALID), (dict(lddh=39), INVALID), (dict(lddx=39), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(ws=None), INVALID), (dict(ws=ODD), INVALID), (dict(bytes=159), INVALID),
    (dict(rows=ROWS + 1), UNSUPPORTED), (dict(n=0, dy=None, h=None), OK), (dict(dx=None, dw=None), OK)])
def test_gradient_refusals(change, status):
    c = dict(rows=4, n=40, dtype=BF16, weight_dtype=F32, eps=1e-6, lddy=40, ldh=40, lddh=40, lddx=40, dy=A, h=A, w=A, dh=A, dx=A, dw=A,
             ws=A, bytes=1 << 40)
    c.update(change)
    p = _lib.NormRmsGrad(*(c[f] for f, _ in _lib.NormRmsGrad._fields_))
    args = [c[f] for f in ("dy", "h", "w", "dh", "dx", "dw", "ws", "bytes")]
    assert spt.lib().norm_rms_grad_run(ctypes.byref(p), *args, None) == status
    assert spt.lib().norm_rms_grad_run(None, *args, None) == INVALID
    assert spt.lib().norm_rms_grad_workspace_bytes(ctypes.byref(p), 1, None) == INVALID


@pytest.mark.parametrize("rows", [0, 1, 255, 5000, 100_000, ROWS])
@pytest.mark.parametrize("n", [1, 200, 513, 8192, 16385, 40000, 2**24])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_gradient_workspace(rows, n, dtype):
    """Planes of dweight: one for a compute unit or more, in step with the workgroups that fit them, whatever the rows."""
    p = _lib.NormRmsGrad(rows, n, dtype, F32, 1e-6, n, n, n, n)
    assert _lib.norm_rms_grad_workspace_bytes(p, False) == 0
    planes, rest = divmod(_lib.norm_rms_grad_workspace_bytes(p, True), 4 * n)
    assert rest == 0 and min(rows, 1) <= planes <= min(rows, 256 * 10)


# -------------------------------------------------------------------------------------- the torch face

def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def bytes_(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


X, W, R, C, S = host(4, 40), host(40), host(4, 40), bytes_(4, 40), bytes_(4, 2)


@pytest.mark.parametrize("call,error,text", [
    (lambda: spt.quantize_mx(X), ValueError, "device tensor"), (lambda: spt.quantize_mx(X.double()), TypeError, "dtype"),
    (lambda: spt.quantize_mx(X, bits=6), ValueError, "bits"), (lambda: spt.pack_mx(C, S, 8), ValueError, "device tensor"),
    (lambda: spt.pack_mx(C.int(), S, 8), ValueError, "bytes"), (lambda: spt.pack_mx(C, S, 5), ValueError, "bits"),
    (lambda: spt.rms_norm(X), ValueError, "device tensor"), (lambda: spt.rms_norm(X.long()), TypeError, "dtype"),
    (lambda: spt.rms_norm_mx(X), ValueError, "device tensor"), (lambda: spt.rms_norm_mx(X, bits=16), ValueError, "bits"),
    (lambda: spt.rms_norm_grad(X, X), ValueError, "device tensor"), (lambda: spt.rms_norm_grad(X, X.int()), TypeError, "dtype"),
    (lambda: spt.MXTensor(bytes_(4, 128), bytes_(1, 4, 64), 8, 4, 40, torch.bfloat16), ValueError, "device tensor"),
    (lambda: spt.MXTensor(bytes_(4, 120), bytes_(1, 4, 64), 8, 4, 40, torch.bfloat16), ValueError, "codes must be"),
    (lambda: spt.MXTensor(bytes_(4, 128), bytes_(4, 64), 8, 4, 40, torch.bfloat16), ValueError, "scales must be"),
    (lambda: spt.MXTensor(bytes_(4, 128), bytes_(1, 4, 64), 7, 4, 40, torch.bfloat16), spt.GemmError, "mx_bytes")])
def test_refusals_of_the_torch_face(call, error, text):
    with pytest.raises(error, match=text):
        call()


def test_tensors_that_require_grad():
    x, w = X.clone().requires_grad_(), W.clone().requires_grad_()
    for call in (lambda: spt.quantize_mx(x), lambda: spt.rms_norm_mx(x), lambda: spt.rms_norm_mx(X, w)):
        with pytest.raises(ValueError, match="no gradient|device tensor"):
            call()
    for call in (lambda: spt.rms_norm(x, out=X.clone()), lambda: spt.rms_norm(X, w, out=X.clone()),
                 lambda: spt.rms_norm(X, residual=x, residual_out=X.clone()), lambda: spt.rms_norm(X, out=x)):
        with pytest.raises(ValueError, match="no part in autograd"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            call()


def test_tensors_with_a_tangent():
    calls = [lambda d: spt.rms_norm(d), lambda d: spt.rms_norm(X, residual=d), lambda d: spt.rms_norm(X, out=d),
             lambda d: spt.rms_norm_grad(d, X), lambda d: spt.rms_norm_grad(X, d), lambda d: spt.rms_norm_grad(X, X, dh=d),
             lambda d: spt.rms_norm_mx(d), lambda d: spt.rms_norm_mx(X, residual=d)]
    for call in calls:
        with forward_ad.dual_level(), torch.no_grad():
            with pytest.raises(ValueError, match="forward-mode"):
                call(forward_ad.make_dual(X, torch.ones_like(X)))
            with pytest.raises(ValueError, match="device tensor"):
                call(X)
