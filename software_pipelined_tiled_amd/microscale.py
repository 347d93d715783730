"""torch-tensor face of include/microscale.h: microscaled tensors (values in 8 or 4 bits with a power of two for each 32
neighbours of a row), their products, and the root-mean-square norm, which writes them or feeds a training step. torch
provides device memory, streams and the autograd graph; all arithmetic runs in the HIP kernels.

Every call enqueues on its tensors' device, on that device's current stream, and synchronises nothing. Workspaces come
from torch's allocator, so calls on several streams, or captured into several graphs, never share one. Rows of a
tensor may be any distance apart (unit column stride). Outputs must not overlap an operand, except where a call names it.

``rms_norm`` is differentiable once, in reverse mode; ``rms_norm_grad`` is the same gradient as a plain call, for
programs that keep no autograd graph and for steps captured into a HIP graph (under ``torch.no_grad()``). The microscaled
formats have no gradient: calls that make or multiply them refuse tensors that require grad, and all refuse operands with
a forward-mode tangent.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .experts import (_16BIT, _CODES, _FLOATS, _enqueue, _matrix, _need, _on_device, _out, _ptr, _rows_apart, _type, _workspace)


def _wants_grad(*tensors) -> bool:
    """Whether these operands make the call part of a graph; operands with a tangent are refused."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("the microscaled operators and the norm have no forward-mode derivative; pass the primal "
                                 "(torch.autograd.forward_ad.unpack_dual)")
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _no_grad(call: str, *tensors) -> None:
    if _wants_grad(*tensors):
        raise ValueError(f"{call} has no gradient; call under torch.no_grad()")


# ------------------------------------------------------------------------------- microscaled tensors

_MX_ROWS, _MX_K = 2**31 - 64, 2**22  # the library's limits


class MXTensor:
    """A microscaled tensor [rows, k] (made by ``quantize_mx``, ``pack_mx`` or ``rms_norm_mx``). bits: 8 (e4m3) or 4
    (e2m1). codes [rows, bytes], rows of whole 128 values, and scales [ceil(rows / 64), blocks, 64], the exponents of the
    scales with a bias of 127 (255: NaN). Codes and scales given here must be zeros behind k, and scales behind the last row: the products
    read them. dtype: what it was made from, the products' default result. It may be pickled, and loaded where there is
    no GPU; every call needs it on one (``to``)."""
    __slots__ = ("bits", "rows", "k", "dtype", "device", "codes_ptr", "scales_ptr", "_data", "_codes", "_scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bits: int, rows: int, k: int, dtype: torch.dtype):
        self._hold(codes, scales, bits, rows, k, dtype)
        if codes.data_ptr() % 16 or scales.data_ptr() % 16:
            raise ValueError("codes and scales must begin on 16 bytes")
        _on_device("codes scales", codes, scales)

    def _hold(self, codes, scales, bits, rows, k, dtype):
        _lib.mx_bytes(rows, k, bits)
        for name, t, shape in zip(("codes", "scales"), (codes, scales), _shapes(rows, k, bits)):
            if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous bytes {shape}")
        if dtype not in _FLOATS:
            raise TypeError(f"unsupported dtype {dtype}")
        self.bits, self.rows, self.k, self.dtype, self.device = bits, rows, k, dtype, codes.device
        self.codes_ptr, self.scales_ptr = codes.data_ptr(), scales.data_ptr()
        self._data, self._codes, self._scales = None, codes, scales
        return self

    def to(self, device) -> MXTensor:
        """Itself where it is on ``device``, else a copy there."""
        codes = self.codes.to(device)
        if codes.device == self.device:
            return self
        parts = codes, self.scales.to(device), self.bits, self.rows, self.k, self.dtype
        return MXTensor(*parts) if codes.is_cuda else _loaded(*parts)

    @property
    def shape(self) -> tuple[int, int]:
        return self.rows, self.k

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:  # views of the one allocation, made when somebody asks for them
            self._codes = self._data[: self.scales_ptr - self.codes_ptr].view(_shapes(self.rows, self.k, self.bits)[0])
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._data[self.scales_ptr - self.codes_ptr:].view(_shapes(self.rows, self.k, self.bits)[1])
        return self._scales

    def __reduce__(self):  # a copy's addresses are its own tensors'
        return _loaded, (self.codes, self.scales, self.bits, self.rows, self.k, self.dtype)

    def __repr__(self) -> str:
        return f"MXTensor({self.rows} x {self.k}, {self.bits} bits, {self.device})"


def _loaded(codes, scales, bits, rows, k, dtype) -> MXTensor:
    """One that may lie in host memory."""
    if codes.is_cuda or scales.is_cuda:
        return MXTensor(codes, scales, bits, rows, k, dtype)
    return MXTensor.__new__(MXTensor)._hold(codes, scales, bits, rows, k, dtype)


def _on_gpu(name: str, q: MXTensor) -> None:
    if q.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor; {name}.to(device) moves it")


def _shapes(rows: int, k: int, bits: int):
    blocks = (k + 127) // 128 * 4
    return (rows, blocks * 4 * bits), ((rows + 63) // 64, blocks, 64)


def _mx_bytes(rows: int, k: int, bits: int) -> tuple[int, int]:
    """Bytes of the codes, a multiple of 16, and of the scales."""
    blocks = (k + 127) // 128 * 4
    return rows * blocks * 4 * bits, ((rows + 63) // 64) * blocks * 64


def _new_mx(rows: int, k: int, bits: int, dtype, device) -> MXTensor:
    """Without the checks: made to the layout here, in one allocation."""
    if rows > _MX_ROWS or k > _MX_K:
        _lib.mx_bytes(rows, k, bits)  # refuses it
    codes, scales = _mx_bytes(rows, k, bits)
    q = MXTensor.__new__(MXTensor)
    q._data = data = torch.empty(codes + scales, dtype=torch.uint8, device=device)
    q.bits, q.rows, q.k, q.dtype, q.device = bits, rows, k, dtype, device
    q.codes_ptr = data.data_ptr()
    q.scales_ptr = q.codes_ptr + codes
    q._codes = q._scales = None
    return q


def _bits(bits) -> int:
    if bits != 8 and bits != 4:
        raise ValueError("bits must be 8 or 4")
    return int(bits)


def quantize_mx(x: torch.Tensor, bits: int = 8) -> MXTensor:
    """x [rows, k] (fp16, bf16 or fp32) in 8 or 4 bits. A block's scale is 2 to the floor of log2 of its largest magnitude,
    less the format's largest exponent (8, or 2); values are rounded to the nearest in units of it, ties to the even
    code, and held to the format's largest (448, or 6). A block with an infinity or a NaN becomes NaN. No gradient."""
    code, bits = _type("x", x, _FLOATS), _bits(bits)
    _on_device("x", x)
    _no_grad("quantize_mx", x)
    ldx = _matrix("x", x)
    rows, k = x.shape
    q = _new_mx(rows, k, bits, x.dtype, x.device)
    _enqueue(x.device, "mx_quantize", x.data_ptr(), code, rows, k, ldx, bits, q.codes_ptr, q.scales_ptr)
    return q


def dequantize_mx(q: MXTensor, dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of ``q``, [rows, k] in fp16, bf16 or fp32 (default: what it was made from), rounded once."""
    _on_gpu("q", q)
    dtype = dtype or (q.dtype if out is None else out.dtype)
    code = _result_code(dtype)
    if out is not None:
        _no_grad("dequantize_mx", out)
    out, ldo, fresh = _out(out, q.rows, q.k, dtype, q.device)
    _enqueue(q.device, "mx_dequantize", q.codes_ptr, q.scales_ptr, q.bits, q.rows, q.k, out.data_ptr(),
             code, ldo)
    if not fresh:
        increment_version(out)
    return out


def pack_mx(codes: torch.Tensor, scales: torch.Tensor, bits: int, k: int | None = None,
            dtype: torch.dtype = torch.bfloat16) -> MXTensor:
    """Lay out a checkpoint's rows: codes [rows, ceil(k * bits / 8)] bytes (of two 4-bit values the first in the low
    half; 8-bit ones may be float8_e4m3fn), scales [rows, ceil(k / 32)] bytes, exponents with a bias of 127. k: by
    default all that the codes hold. ``dtype``: the products' default result. No gradient."""
    bits = _bits(bits)
    _no_grad("pack_mx", codes, scales)  # of the 8-bit types: a view as bytes drops out of the graph
    if bits == 8 and codes.dtype == torch.float8_e4m3fn:
        codes = codes.view(torch.uint8)
    if scales.dtype == torch.float8_e8m0fnu:
        scales = scales.view(torch.uint8)
    _need(codes.dtype == torch.uint8 and scales.dtype == torch.uint8, "codes and scales must be bytes")
    _on_device("codes scales", codes, scales)
    _type("the result", torch.empty(0, dtype=dtype), _FLOATS)
    ldc = _matrix("codes", codes)
    rows = codes.shape[0]
    k = codes.shape[1] * 8 // bits if k is None else int(k)
    _need(k >= 0 and codes.shape[1] == -(-k * bits // 8), f"codes must have {-(-k * bits // 8)} bytes a row")
    lds = _matrix("scales", scales, rows, -(-k // 32))
    q = _new_mx(rows, k, bits, dtype, codes.device)
    _enqueue(codes.device, "mx_pack", codes.data_ptr(), ldc, scales.data_ptr(), lds, bits, rows, k, q.codes_ptr,
             q.scales_ptr)
    return q


def mx_matmul(a: MXTensor, b: MXTensor, out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A·Bᵀ [m, n] of A [m, k] and B [n, k]: 8 x 8, 4 x 4, or 8-bit rows with a 4-bit B. fp16, bf16 (default: A's
    ``dtype``) or fp32 results from fp32 sums, rounded once. 16-bit results come from the matrix cores' own formats, which for
    8-bit operands keep 13 bits below the largest of the products they add at a time, far below the result's rounding; fp32
    results of 8-bit operands go through bf16 instructions, whose sums keep all of fp32, at less than half the rate. No
    gradient."""
    dev = a.device
    _on_gpu("a", a)
    if a.k != b.k:
        raise ValueError(f"a has rows of {a.k}, b of {b.k}")
    if b.device != dev:
        raise ValueError(f"b is on {b.device}, a on {dev}")
    _need(a.bits == 8 or b.bits == 4, "a 4-bit a goes with a 4-bit b")
    if out is not None:
        _no_grad("mx_matmul", out)
    dtype = out_dtype or (a.dtype if out is None else out.dtype)
    code = _result_code(dtype)
    out, ldc, fresh = _out(out, a.rows, b.rows, dtype, dev)
    p = _lib.GemmMx(a.rows, b.rows, a.k, a.bits, b.bits, code, ldc)
    ws_bytes = _lib.gemm_mx_workspace_bytes(p)
    ws = _workspace(ws_bytes, dev)
    _enqueue(dev, "gemm_mx_run", p, a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, out.data_ptr(), _ptr(ws), ws_bytes)
    if not fresh:
        increment_version(out)
    return out


def _result_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def mx_linear(x: torch.Tensor, w: MXTensor, bits: int = 8, out_dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """x [rows, k] quantised to ``bits`` and multiplied with the weight w [n, k]: [rows, n] in x's type or ``out_dtype``.
    The same as ``mx_matmul(quantize_mx(x, bits), w)``, with one workspace, and with its sums: ``out_dtype=torch.float32`` keeps all
    of fp32 in those of 8-bit rows. A 4-bit weight takes rows of 8 bits or 4, an 8-bit one rows of 8. No gradient."""
    code, bits, dev = _type("x", x, _FLOATS), _bits(bits), x.device
    _need(bits == 8 or w.bits == 4, "rows of 4 bits go with a 4-bit weight")
    if not x.is_cuda or w.device != dev:
        _on_device("x w", x, w.codes)
    _no_grad("mx_linear", x, out)
    ldx = _matrix("x", x, None, w.k)
    rows, k = x.shape
    dtype = out_dtype or (x.dtype if out is None else out.dtype)
    out_code = _result_code(dtype)
    out, ldc, fresh = _out(out, rows, w.rows, dtype, dev)
    p = _lib.GemmMx(rows, w.rows, k, bits, w.bits, out_code, ldc)
    ws_bytes = _lib.gemm_mx_workspace_bytes(p)
    codes, scales = _mx_bytes(rows, k, bits)
    ws = torch.empty(codes + scales + ws_bytes, dtype=torch.uint8, device=dev)  # each part a multiple of 16 bytes long
    at = ws.data_ptr()
    _enqueue(dev, "mx_quantize", x.data_ptr(), code, rows, k, ldx, bits, at, at + codes)
    _enqueue(dev, "gemm_mx_run", p, at, at + codes, w.codes_ptr, w.scales_ptr, out.data_ptr(), at + codes + scales, ws_bytes)
    if not fresh:
        increment_version(out)
    return out


# ------------------------------------------------------------------------------- norm

def _norm_weight(weight, x):
    """The weight, contiguous, and its type's code."""
    if weight is None:
        return None, 0
    code = _type("weight", weight, _FLOATS)
    if weight.dim() != 1 or weight.shape[0] != x.shape[1]:
        raise ValueError(f"weight must be [{x.shape[1]}]")
    return weight.contiguous(), code


def _eps(eps) -> float:
    eps = float(eps)
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps must be a number from 0 on")
    return eps


def _norm_args(x, weight, residual, eps, residual_out):
    """Checks what both norms take; h is x's own where there is no residual."""
    code = _type("x", x, _FLOATS)
    _on_device("x weight residual", x, weight, residual)
    ldx = _matrix("x", x)
    rows, n = x.shape
    weight, wcode = _norm_weight(weight, x)
    eps = _eps(eps)
    if residual is None:
        _need(residual_out is None, "residual_out goes with a residual")
        return _lib.NormRms(rows, n, code, wcode, eps, ldx, 0, 0, 0), weight, None, True
    _need(residual.dtype == x.dtype, "residual must have x's dtype")
    ldr = _matrix("residual", residual, rows, n)
    h, ldh, fresh = _out(residual_out, rows, n, x.dtype, x.device)
    return _lib.NormRms(rows, n, code, wcode, eps, ldx, ldr, ldh, 0), weight, h, fresh


def _norm(x, weight, eps, residual, out, residual_out):
    p, weight, h, h_fresh = _norm_args(x, weight, residual, eps, residual_out)
    y, p.ldy, fresh = _out(out, p.rows, p.n, x.dtype, x.device)
    _enqueue(x.device, "norm_rms_run", p, x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(h), y.data_ptr())
    if not fresh:
        increment_version(y)
    if not h_fresh:
        increment_version(h)
    return y, h


def _norm_grad(dy, h, weight, eps, dh, want_dx=True, want_dw=True):
    code = _type("h", h, _FLOATS)
    _on_device("h dy weight dh", h, dy, weight, dh)
    _need(dy.dtype == h.dtype and (dh is None or dh.dtype == h.dtype), "dy and dh must have h's dtype")
    ldh = _matrix("h", h)
    rows, n = h.shape
    lddy = _matrix("dy", dy, rows, n)
    lddh = _matrix("dh", dh, rows, n) if dh is not None else 0
    weight, wcode = _norm_weight(weight, h)
    dx = torch.empty(rows, n, dtype=h.dtype, device=h.device) if want_dx else None
    dw = torch.empty(n, dtype=weight.dtype, device=h.device) if want_dw and weight is not None else None
    p = _lib.NormRmsGrad(rows, n, code, wcode, _eps(eps), lddy, ldh, lddh, n)
    ws_bytes = _lib.norm_rms_grad_workspace_bytes(p, dw is not None)
    ws = _workspace(ws_bytes, h.device)
    _enqueue(h.device, "norm_rms_grad_run", p, dy.data_ptr(), h.data_ptr(), _ptr(weight), _ptr(dh), _ptr(dx), _ptr(dw),
             _ptr(ws), ws_bytes)
    return dx, dw


class _OnceGrad(torch.autograd.Function):
    """The gradient of tensors that a graph holds: it stays in the graph, and differentiating it raises there."""
    @staticmethod
    def forward(ctx, dy, h, weight, eps, dh):
        return _norm_grad(dy, h, weight, eps, dh)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("rms_norm is differentiable once; call rms_norm_grad under torch.no_grad() where its result is a "
                           "constant")


def rms_norm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6,
                  dh: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradients of ``rms_norm`` for x (and, the same tensor, for the residual) and for the weight (None without one),
    in h's and the weight's types. h: what was normalised, x itself without a residual; dh: the gradient that reaches the
    returned h by itself."""
    if _wants_grad(dy, h, weight, dh):
        return _OnceGrad.apply(dy, h, weight, eps, dh)
    return _norm_grad(dy, h, weight, eps, dh)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        ctx.set_materialize_grads(False)
        ctx.eps = eps
        y, h = _norm(x, weight, eps, residual, None, None)
        ctx.save_for_backward(x if h is None else h, weight)
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        want_x, want_w, _, want_r = ctx.needs_input_grad
        if dy is None:  # y was not used: what reached h passes on
            return dh if want_x else None, None, None, dh if want_r else None
        _wants_grad(dy, dh)  # refuses tangents
        dx, dw = _norm_grad(_rows_apart(dy), h, weight, ctx.eps, None if dh is None else _rows_apart(dh), want_x or want_r,
                            want_w)
        return dx if want_x else None, dw, None, dx if want_r else None


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, residual: torch.Tensor | None = None,
             out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of x [rows, n] (fp16, bf16 or fp32), in x's type; h = x, and
    the result is y. With a ``residual`` of x's shape and type h = x + residual, rounded to that type, and the result is
    (y, h). weight [n] fp16, bf16 or fp32, or None for ones. Statistics and products are fp32, y is rounded once; the sum
    of a row's squares has to stay inside fp32's range. ``out`` may be x, ``residual_out`` x or residual, and the two need
    memory of their own; with either the call takes no part in autograd."""
    if out is not None or residual_out is not None:
        _need(out is None or residual_out is None or out.data_ptr() != residual_out.data_ptr() or not out.numel(),
              "out and residual_out need memory of their own")
        _need(not _wants_grad(x, weight, residual, out, residual_out),
              "out= and residual_out= take no part in autograd; call under torch.no_grad()")
    elif _wants_grad(x, weight, residual):
        return _Norm.apply(x, weight, eps, residual)
    y, h = _norm(x, weight, eps, residual, out, residual_out)
    return y if residual is None else (y, h)


def rms_norm_mx(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, residual: torch.Tensor | None = None,
                bits: int = 8, residual_out: torch.Tensor | None = None):
    """``rms_norm`` with y quantised to 8 or 4 bits from its fp32 values, as ``quantize_mx`` does it: an ``MXTensor`` for
    ``mx_matmul``, or (that, h) with a residual. No gradient."""
    bits = _bits(bits)
    _no_grad("rms_norm_mx", x, weight, residual, residual_out)
    p, weight, h, h_fresh = _norm_args(x, weight, residual, eps, residual_out)
    q = _new_mx(p.rows, p.n, bits, x.dtype, x.device)
    _enqueue(x.device, "norm_rms_mx_run", p, bits, x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(h), q.codes_ptr,
             q.scales_ptr)
    if not h_fresh:
        increment_version(h)
    return q if residual is None else (q, h)
