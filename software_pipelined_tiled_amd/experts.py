"""torch-tensor face of include/experts.h: tokens sorted by expert and back, the experts' products with
their gradients, and products with 4-bit weights. torch provides device memory, streams and the
autograd graph; all arithmetic runs in the HIP kernels.

Every call enqueues on its tensors' device, on that device's current stream, and synchronises nothing.
Workspaces come from torch's allocator, so calls on several streams, or captured into several graphs,
never share one. Rows of a tensor may be any distance apart (unit column stride). ``out`` must not overlap an
operand: kernels read and write at once.

``gather_rows``, ``combine_rows``, ``grouped_matmul`` and ``routed_matmul`` are differentiable once, in reverse mode;
operands with a forward-mode tangent are refused. The ``*_grad`` functions are the same gradients as plain calls, for
programs that keep no autograd graph; of tensors that require grad they stay in the graph, where differentiating them
raises. A training step captured into a HIP graph is safest with those, under ``torch.no_grad()``: while an eager graph of
the same leaves is alive (a result that stayed in it will do), torch's backward ties a capture to that graph's stream and
ends the process.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .torch_api import dtype_code

_16BIT = (torch.float16, torch.bfloat16)
_FLOATS = (*_16BIT, torch.float32)
_SORT_ONE = 4096  # slots that one workgroup sorts without a workspace
_CODES = {t: dtype_code(t) for t in _FLOATS}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# ------------------------------------------------------------------------------------ arguments
# These calls are a few microseconds of GPU work in a decoding loop: the checks cost what they have to,
# messages are put together only for a refusal, and the device is switched only where it is another.

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on_device(names: str, first: torch.Tensor, *others) -> None:
    """Device tensors, all on the first one's device (None: an operand that is not there)."""
    device = first.device
    if first.is_cuda:
        for t in others:
            if t is not None and t.device != device:
                break
        else:
            return
    for name, t in zip(names.split(), (first, *others)):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other operands on {device}")


def _matrix(name: str, t: torch.Tensor, rows: int | None = None, cols: int | None = None) -> int:
    """Checks a 2-d operand and returns its row stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    r, c = t.shape
    if rows is not None and r != rows:
        raise ValueError(f"{name} must have {rows} rows, has {r}")
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns, has {c}")
    if t.is_contiguous():
        return c
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    if r <= 1:
        return c
    ld = t.stride(0)
    if ld < c:
        raise ValueError(f"{name} must be row-major with rows that do not overlap")
    return ld


def _stack(name: str, t: torch.Tensor) -> tuple[int, int, int, int, int]:
    """Checks a [experts, n, k] operand and returns its sizes, row stride and expert stride."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions [experts, n, k]")
    e, n, k = t.shape
    if k > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    ld = t.stride(1) if n > 1 else k
    if ld < k:
        raise ValueError(f"{name}'s rows must not overlap")
    stride = t.stride(0) if e > 1 else n * ld
    if n > 0 and stride < (n - 1) * ld + k:
        raise ValueError(f"{name}'s matrices must not overlap")
    return e, n, k, ld, stride


def _rows_apart(t: torch.Tensor) -> torch.Tensor:
    """A gradient as autograd hands it over may be a broadcast or transposed view."""
    r, c = t.shape[-2:]
    ok = (c <= 1 or t.stride(-1) == 1) and (r <= 1 or t.stride(-2) >= c)
    return t if ok else t.contiguous()


def _offsets(offsets: torch.Tensor, experts: int) -> None:
    if (offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] != experts + 1
            or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be {experts + 1} contiguous 32-bit integers")


def _type(name: str, t: torch.Tensor, kinds) -> int:
    dtype = t.dtype
    if dtype not in kinds:
        raise TypeError(f"unsupported dtype {dtype} of {name}")
    return _CODES[dtype]


def _refuse_tangents(tensors) -> None:
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("the experts' operators have no forward-mode derivative; pass the primal "
                             "(torch.autograd.forward_ad.unpack_dual)")


def _wants_grad(*tensors) -> bool:
    """Whether these operands make the call part of a graph. Every call asks, so that operands with a tangent, which
    the kernels' results would not carry, are refused here; they exist only inside a dual level."""
    if forward_ad._current_level >= 0:
        _refuse_tangents(tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _out(out, rows: int, cols: int, dtype, device) -> tuple[torch.Tensor, int, bool]:
    """The output, its row stride, and whether it is new (then the rows nobody computes are zeroed). One that is not
    new was written behind torch's back, which ``increment_version`` tells autograd: it may have been saved."""
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device), cols, True
    if out.device != device:
        raise ValueError(f"out is on {out.device}, the operands on {device}")
    if out.dtype != dtype:
        raise ValueError(f"out must be {dtype}")
    return out, _matrix("out", out, rows, cols), False


def _no_autograd(out, *inputs) -> None:
    _need(not _wants_grad(out, *inputs), "out= takes no part in autograd; call under torch.no_grad()")


def _enqueue(device: torch.device, entry: str, *args) -> None:
    """The C entry point `entry`(*args, stream) with `device` current, on its current stream."""
    index, fn = device.index, getattr(_lib.lib(), entry)
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        raise _lib.GemmError(status, entry)


def _workspace(nbytes: int, device: torch.device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


class _Once(torch.autograd.Function):
    """A gradient of tensors that a graph holds: it stays in the graph, and differentiating it raises there instead of
    leaving a term out."""
    @staticmethod
    def forward(ctx, gradient, *args):
        return gradient(*args)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the experts' operators are differentiable once; call their gradients under torch.no_grad() "
                           "where they are constants")


# ---------------------------------------------------------------------------- tokens by expert

class TokenOrder:
    """A router's choices sorted by expert (made by ``sort_tokens``).

    offsets [num_experts + 1]: expert e owns sorted rows offsets[e] .. offsets[e + 1]; the last entry is
    the number of kept slots. slots [tokens * top_k]: sorted position to slot (token * top_k + j).
    rows [tokens, top_k]: slot to sorted position. All 32-bit.
    """
    __slots__ = ("offsets", "slots", "rows", "num_experts", "tokens", "top_k", "sorted_rows")

    def __init__(self, offsets: torch.Tensor, slots: torch.Tensor, rows: torch.Tensor, num_experts: int):
        _need(rows.dim() == 2, "rows must be [tokens, top_k]")
        for name, t, size in (("offsets", offsets, num_experts + 1), ("slots", slots, rows.numel()),
                              ("rows", rows, rows.numel())):
            if t.dtype != torch.int32 or t.numel() != size or not t.is_contiguous() or t.device != rows.device:
                raise ValueError(f"{name} must be {size} contiguous 32-bit integers on rows' device")
        self._set(offsets, slots, rows, num_experts)

    def _set(self, offsets, slots, rows, num_experts):
        self.offsets, self.slots, self.rows, self.num_experts = offsets, slots, rows, num_experts
        self.tokens, self.top_k = rows.shape
        self.sorted_rows = self.tokens * self.top_k
        return self

    @property
    def kept_ptr(self) -> int:
        """Where offsets[num_experts] lies."""
        return self.offsets.data_ptr() + 4 * self.num_experts


def sort_tokens(experts: torch.Tensor, num_experts: int) -> TokenOrder:
    """Sort the slots of ``experts`` ([tokens, top_k] or [tokens] ids, 32- or 64-bit integers) by expert,
    slots of one expert in their own order. Ids outside [0, num_experts) are dropped: they sort behind
    the last expert. At most 1024 experts."""
    bits = 64 if experts.dtype == torch.int64 else 32
    if bits == 32 and experts.dtype != torch.int32:
        raise TypeError(f"unsupported dtype {experts.dtype} of experts")
    if not experts.is_cuda:
        raise ValueError("experts must be a device tensor")
    dim = experts.dim()
    if dim != 2:
        _need(dim == 1, "experts must be [tokens, top_k] or [tokens]")
        experts = experts[:, None]
    num_experts = int(num_experts)
    ids = experts.contiguous()
    n, dev = ids.numel(), ids.device
    ws_bytes = _lib.experts_sort_workspace_bytes(n, num_experts) if n > _SORT_ONE or not 0 < num_experts <= 1024 else 0
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    slots = torch.empty(n, dtype=torch.int32, device=dev)
    rows = torch.empty(ids.shape, dtype=torch.int32, device=dev)
    ws = _workspace(ws_bytes, dev)
    _enqueue(dev, "experts_sort", ids.data_ptr(), bits, n, num_experts, offsets.data_ptr(), slots.data_ptr(),
             rows.data_ptr(), _ptr(ws), ws_bytes)
    return TokenOrder.__new__(TokenOrder)._set(offsets, slots, rows, num_experts)  # nothing to check


def _gather(x, order, out):
    code, rows, dev = _type("x", x, _FLOATS), order.rows, x.device
    if not x.is_cuda or rows.device != dev:
        _on_device("x order", x, rows)
    ldx = _matrix("x", x, order.tokens)
    width = x.shape[1]
    if out is None:
        out, ldo, fresh = x.new_empty((order.sorted_rows, width)), width, True
    else:
        out, ldo, fresh = _out(out, order.sorted_rows, width, x.dtype, dev)
    _enqueue(dev, "experts_gather", x.data_ptr(), code, order.tokens, order.top_k, width, ldx, rows.data_ptr(),
             order.kept_ptr, out.data_ptr(), ldo, fresh)
    if not fresh:
        increment_version(out)
    return out


def _router_weights(weights, order):
    """The weights, contiguous, and their type's code."""
    if weights is None:
        return None, 0
    code = _type("weights", weights, _FLOATS)
    if weights.shape != order.rows.shape:
        raise ValueError(f"weights must be {tuple(order.rows.shape)}")
    return weights.contiguous(), code


def _combine(y, order, weights, out):
    code, rows, dev = _type("y", y, _FLOATS), order.rows, y.device
    if not y.is_cuda or rows.device != dev or (weights is not None and weights.device != dev):
        _on_device("y order weights", y, rows, weights)
    ldy = _matrix("y", y, order.sorted_rows)
    weights, wcode = _router_weights(weights, order)
    width = y.shape[1]
    if out is None:
        out, ldo, fresh = y.new_empty((order.tokens, width)), width, True
    else:
        out, ldo, fresh = _out(out, order.tokens, width, y.dtype, dev)
    _enqueue(dev, "experts_combine", y.data_ptr(), code, order.tokens, order.top_k, width, ldy, rows.data_ptr(),
             order.kept_ptr, _ptr(weights), wcode, out.data_ptr(), ldo)
    if not fresh:
        increment_version(out)
    return out


def gather_rows_grad(dsorted: torch.Tensor, order: TokenOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``gather_rows``: each token's sum over its kept rows of ``dsorted``, in fp32, rounded once."""
    if out is not None:
        _no_autograd(out, dsorted)
    elif _wants_grad(dsorted):
        return _Once.apply(gather_rows_grad, dsorted, order)
    return _combine(dsorted, order, None, out)


def combine_rows_grad(dout: torch.Tensor, y: torch.Tensor, order: TokenOrder,
                      weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradients of ``combine_rows`` for y and the weights (None without weights), in their types. Rows
    and weights of dropped slots get zeros."""
    if _wants_grad(dout, y, weights):
        return _Once.apply(combine_rows_grad, dout, y, order, weights)
    code = _type("y", y, _FLOATS)
    _on_device("y dout order weights", y, dout, order.rows, weights)
    _need(dout.dtype == y.dtype, "dout must have y's dtype")
    width, dev = y.shape[1] if y.dim() == 2 else 0, y.device
    ldy = _matrix("y", y, order.sorted_rows)
    lddo = _matrix("dout", dout, order.tokens, width)
    weights, wcode = _router_weights(weights, order)
    dw = torch.empty(order.rows.shape, dtype=weights.dtype, device=dev) if weights is not None else None
    dy = torch.empty((order.sorted_rows, width), dtype=y.dtype, device=dev)
    _enqueue(dev, "experts_combine_grad", dout.data_ptr(), lddo, y.data_ptr(), code, order.tokens, order.top_k, width,
             ldy, order.rows.data_ptr(), order.kept_ptr, _ptr(weights), wcode, dy.data_ptr(), width, _ptr(dw), True)
    return dy, dw


# A graph keeps an order's tensors where torch watches what it saves: one that is changed before backward raises.

def _saved_order(rows, offsets) -> TokenOrder:
    return TokenOrder.__new__(TokenOrder)._set(offsets, None, rows, offsets.numel() - 1)  # backward needs no slots


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.save_for_backward(order.rows, order.offsets)
        return _gather(x, order, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dsorted):
        return gather_rows_grad(_rows_apart(dsorted), _saved_order(*ctx.saved_tensors)), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, order, weights):
        ctx.save_for_backward(y, weights, order.rows, order.offsets)
        return _combine(y, order, weights, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, weights, rows, offsets = ctx.saved_tensors
        dy, dw = combine_rows_grad(_rows_apart(dout), y, _saved_order(rows, offsets), weights)
        return dy, None, dw


def gather_rows(x: torch.Tensor, order: TokenOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows x [tokens, width] in the order's sorted rows [tokens * top_k, width]. Rows at dropped
    positions are zeros in a new tensor, and left as they were in ``out``."""
    if out is not None:
        _no_autograd(out, x)
    elif _wants_grad(x):
        return _Gather.apply(x, order)
    return _gather(x, order, out)


def combine_rows(y: torch.Tensor, order: TokenOrder, weights: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Each token's weighted sum of its kept sorted rows: y [tokens * top_k, width], weights [tokens,
    top_k] (fp32 or 16-bit; None: ones). Summed in fp32 in the slots' order, rounded once to y's type."""
    if out is not None:
        _no_autograd(out, y, weights)
    elif _wants_grad(y, weights):
        return _Combine.apply(y, order, weights)
    return _combine(y, order, weights, out)


# --------------------------------------------------------------------------- experts' products

def _grouped_run(mode, x, y, out, offsets, rows, experts, n, k, ldx, ldy, ldo, stride, fresh, tile):
    p = _lib.GemmGrouped(mode, rows, experts, n, k, dtype_code(x.dtype), dtype_code(out.dtype), ldx, ldy, ldo, stride,
                         fresh, tile)
    xp, yp = x.data_ptr(), y.data_ptr()
    ws_bytes = _lib.gemm_grouped_workspace_bytes(p, xp, yp)
    ws = _workspace(ws_bytes, x.device)
    _enqueue(x.device, "gemm_grouped_run", p, xp, yp, out.data_ptr(), offsets.data_ptr(), _ptr(ws), ws_bytes)
    if not fresh:
        increment_version(out)
    return out


def _result_type(out_dtype, out, default):
    dtype = out_dtype or (default if out is None else out.dtype)
    dtype_code(dtype)
    return dtype


def _grouped_forward(A, B, offsets, out_dtype, out, tile):
    _type("A", A, _16BIT)
    _need(B.dtype == A.dtype, "B must have A's dtype")
    _on_device("A B offsets", A, B, offsets)
    E, N, K, ldb, stride = _stack("B", B)
    lda = _matrix("A", A, None, K)
    _offsets(offsets, E)
    rows = A.shape[0]
    C, ldc, fresh = _out(out, rows, N, _result_type(out_dtype, out, A.dtype), A.device)
    return _grouped_run(_lib.GEMM_GROUPED_FORWARD, A, B, C, offsets, rows, E, N, K, lda, ldb, ldc, stride, fresh,
                        tile)


def grouped_matmul_grad_a(dC: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                          tile: int = 0) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for A: dA[i] = dC[i]·B[e] for expert e's rows i, dC 16-bit, dA in its type
    whatever the forward's ``out_dtype`` was. Rows of no expert: zeros in a new tensor, left as they were in ``out``."""
    if out is not None:
        _no_autograd(out, dC, B)
    elif _wants_grad(dC, B):
        return _Once.apply(grouped_matmul_grad_a, dC, B, offsets, None, tile)
    _type("dC", dC, _16BIT)
    _need(B.dtype == dC.dtype, "B must have dC's dtype")
    _on_device("dC B offsets", dC, B, offsets)
    E, N, K, ldb, stride = _stack("B", B)
    lddc = _matrix("dC", dC, None, N)
    _offsets(offsets, E)
    rows = dC.shape[0]
    dA, lda, fresh = _out(out, rows, K, dC.dtype, dC.device)
    return _grouped_run(_lib.GEMM_GROUPED_GRAD_A, dC, B, dA, offsets, rows, E, N, K, lddc, ldb, lda, stride, fresh,
                        tile)


def grouped_matmul_grad_b(dC: torch.Tensor, A: torch.Tensor, offsets: torch.Tensor,
                          out_dtype: torch.dtype | None = None, tile: int = 0) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for B, [experts, n, k]: dB[e] = sum over expert e's rows i of
    dC[i]ᵀ·A[i], in A's type or ``out_dtype`` (fp32 for a main copy of the weights); zeros for an expert
    without rows."""
    if _wants_grad(dC, A):
        return _Once.apply(grouped_matmul_grad_b, dC, A, offsets, out_dtype, tile)
    _type("A", A, _16BIT)
    _need(dC.dtype == A.dtype, "dC must have A's dtype")
    _on_device("A dC offsets", A, dC, offsets)
    _need(offsets.dim() == 1 and offsets.shape[0] >= 1, "offsets must be [experts + 1]")
    E = offsets.shape[0] - 1
    _offsets(offsets, E)
    lda = _matrix("A", A)
    rows, K = A.shape
    lddc = _matrix("dC", dC, rows)
    N = dC.shape[1]
    dB = torch.empty((E, N, K), dtype=_result_type(out_dtype, None, A.dtype), device=A.device)
    return _grouped_run(_lib.GEMM_GROUPED_GRAD_B, dC, A, dB, offsets, rows, E, N, K, lddc, lda, K, N * K, True,
                        tile)


class _Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B, offsets, out_dtype, tile):
        ctx.save_for_backward(A, B, offsets)
        return _grouped_forward(A, B, offsets, out_dtype, None, tile)

    @staticmethod
    @once_differentiable
    def backward(ctx, dC):
        A, B, offsets = ctx.saved_tensors
        dC = _rows_apart(dC.to(A.dtype))  # the products take 16-bit operands of one type: fp32 loses range and bits
        dA = grouped_matmul_grad_a(dC, B, offsets) if ctx.needs_input_grad[0] else None
        dB = grouped_matmul_grad_b(dC, A, offsets) if ctx.needs_input_grad[1] else None
        return dA, dB, None, None, None


def grouped_matmul(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, out_dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None, tile: int = 0) -> torch.Tensor:
    """C[i] = A[i]·B[e]ᵀ for expert e's rows offsets[e] <= i < offsets[e + 1]: A [rows, k] and B [experts, n, k]
    fp16 or bf16, fp32 sums, C in A's type or ``out_dtype``. ``offsets``: 32-bit, ascending, on the device: a
    ``TokenOrder``'s, or its [lo : hi + 1] with B of experts lo .. hi - 1. Rows of no expert, behind the last or in
    front of the first, are zeros in a new tensor, left as they were in ``out``. ``tile``: rows of an output
    tile, 0 for the library's choice, else 32, 128 or 256 (the same sums, in fp32, which 32-row tiles may add in
    parts).

    Gradients: the products take 16-bit operands, so a dC that arrives in fp32 (``out_dtype``) is rounded to A's type
    first, and dA and dB come in it. With fp16 operands a gradient above 65504 becomes infinite and one below 2^-25
    zero: scale the loss, or take bf16."""
    if out is not None:
        _no_autograd(out, A, B)
    elif _wants_grad(A, B):
        return _Grouped.apply(A, B, offsets, out_dtype, tile)
    return _grouped_forward(A, B, offsets, out_dtype, out, tile)


# ------------------------------------------------------------------------------- 4-bit weights

@dataclass(frozen=True)
class W4Weight:
    """4-bit weights laid out for ``w4_matmul`` (made by ``pack_w4``). ``stacked``: from
    [experts, n, k], for rows sorted by expert; else one [n, k] weight."""
    packed: torch.Tensor
    matrices: int
    stacked: bool
    n: int
    k: int
    group_size: int
    has_zeros: bool
    dtype: torch.dtype

    def __post_init__(self):
        nbytes = _lib.gemm_w4_packed_bytes(self.matrices, self.n, self.k, self.group_size, self.has_zeros)
        p = self.packed
        _need(p.dtype == torch.uint8 and p.is_contiguous() and p.numel() == nbytes and (self.stacked or self.matrices == 1),
              f"packed must be {nbytes} contiguous bytes from pack_w4")


def pack_w4(q: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
            group_size: int = 128) -> W4Weight:
    """Lay out weights (q - z) * s: q [n, k] or [experts, n, k] bytes holding 0 .. 15 (the low four bits are
    taken), scales [..., n, ceil(k / group_size)] fp16 or bf16 (the products' type), zeros bytes of the same
    shape, or None for z = 8. group_size 32, 64 or 128. No gradient for the scales."""
    _need(not _wants_grad(scales), "pack_w4 has no gradient for the scales; call under torch.no_grad()")
    _need(q.dtype == torch.uint8 and q.dim() in (2, 3), "q must be [n, k] or [experts, n, k] bytes")
    _type("scales", scales, _16BIT)
    _on_device("q scales zeros", q, scales, zeros)
    group_size = int(group_size)
    _need(group_size in (32, 64, 128), "group_size must be 32, 64 or 128")
    n, k = q.shape[-2:]
    shape = (*q.shape[:-1], -(-k // group_size))
    _need(tuple(scales.shape) == shape, f"scales must be {shape}")
    _need(zeros is None or (zeros.dtype == torch.uint8 and tuple(zeros.shape) == shape), f"zeros must be bytes {shape}")
    matrices = q.shape[0] if q.dim() == 3 else 1
    nbytes = _lib.gemm_w4_packed_bytes(matrices, n, k, group_size, zeros is not None)
    q, scales = q.contiguous(), scales.contiguous()
    zeros = zeros.contiguous() if zeros is not None else None
    packed = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _enqueue(q.device, "gemm_w4_pack", q.data_ptr(), scales.data_ptr(), _ptr(zeros), matrices, n, k, group_size,
             packed.data_ptr())
    return W4Weight(packed, matrices, q.dim() == 3, n, k, group_size, zeros is not None, scales.dtype)


def w4_matmul(x: torch.Tensor, w: W4Weight, offsets: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """x [rows, k] times the 4-bit weight, [rows, n]: one weight for all rows, or expert e's for rows
    offsets[e] <= i < offsets[e + 1] of a weight packed from [experts, n, k]. x in the scales' type; no weight
    is rounded, sums are fp32. No gradient. Rows of no expert, behind the last or in front of the first, are zeros
    in a new tensor, left as they were in ``out``."""
    code = _type("x", x, _16BIT)
    _need(x.dtype == w.dtype, "x must have the dtype of the scales")
    _on_device("x weight offsets", x, w.packed, offsets)
    _need((offsets is not None) == w.stacked, "offsets go with a weight packed from [experts, n, k], and only with one")
    _need(not _wants_grad(x, out), "w4_matmul has no gradient; call under torch.no_grad()")
    ldx = _matrix("x", x, None, w.k)
    if offsets is not None:
        _offsets(offsets, w.matrices)
    rows, dev = x.shape[0], x.device
    dtype = _result_type(out_dtype, out, x.dtype)
    out, ldo, fresh = _out(out, rows, w.n, dtype, dev)
    p = _lib.GemmW4(rows, w.matrices, w.n, w.k, w.group_size, w.has_zeros, code, dtype_code(dtype), ldx, ldo, fresh)
    ws_bytes = _lib.gemm_w4_workspace_bytes(p, offsets is not None)
    ws = _workspace(ws_bytes, dev)
    _enqueue(dev, "gemm_w4_run", p, x.data_ptr(), w.packed.data_ptr(), _ptr(offsets), out.data_ptr(), _ptr(ws), ws_bytes)
    if not fresh:
        increment_version(out)
    return out


# --------------------------------------------------------------------------------- all together

def routed_matmul(x: torch.Tensor, weight: torch.Tensor | W4Weight, experts: torch.Tensor,
                  weights: torch.Tensor | None = None) -> torch.Tensor:
    """A routed linear layer: out[t] = sum over j of weights[t, j] * x[t]·B[experts[t, j]]ᵀ, with B
    [experts, n, k] 16-bit, or packed in 4 bits (no gradient then). The tokens are sorted by expert, their
    rows gathered, multiplied and combined; ids outside the experts are dropped. The experts' outputs are rounded to
    x's 16-bit type before the weighted sum, which is fp32 and rounded again (half the bytes between the two kernels;
    ``grouped_matmul`` with ``out_dtype=torch.float32`` and ``combine_rows`` keep them in fp32). Differentiable in x, B
    and the weights."""
    four_bits = isinstance(weight, W4Weight)
    _need(four_bits or weight.dim() == 3, "the weight must be [experts, n, k]")
    num = weight.matrices if four_bits else weight.shape[0]
    _need(not four_bits or weight.stacked, "the weight must be packed from [experts, n, k]")
    _need(x.dim() == 2 and experts.dim() in (1, 2), "x must be [tokens, k], experts [tokens, top_k] or [tokens]")
    _need(experts.shape[0] == x.shape[0], f"experts must have {x.shape[0]} rows")
    order = sort_tokens(experts, num)
    rows = gather_rows(x, order)
    y = w4_matmul(rows, weight, order.offsets) if four_bits else grouped_matmul(rows, weight, order.offsets)
    if weights is not None and weights.dim() == 1:
        weights = weights[:, None]
    return combine_rows(y, order, weights)
