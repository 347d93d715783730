"""torch-tensor face of include/experts.h: tokens sorted by expert and back, the experts' products with
their gradients, and products with 4-bit weights. torch provides device memory, streams and the
autograd graph; all arithmetic runs in the HIP kernels.

Every call enqueues on its tensors' device, on that device's current stream, and synchronises nothing.
Workspaces come from torch's allocator, so calls on several streams, or captured into several graphs,
never share one. Rows of a tensor may be any distance apart (unit column stride).

``gather_rows``, ``combine_rows``, ``grouped_matmul`` and ``routed_matmul`` are differentiable once. The
``*_grad`` functions are the same gradients as plain calls, for programs that keep no autograd graph (a
training step captured into a HIP graph among them).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .torch_api import dtype_code

_16BIT = (torch.float16, torch.bfloat16)


# ------------------------------------------------------------------------------------ arguments

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None:
            _need(t.is_cuda, f"{name} must be a device tensor")
            _need(t.device == device, f"{name} is on {t.device}, the other operands on {device}")


def _matrix(name: str, t: torch.Tensor, rows: int | None = None, cols: int | None = None) -> int:
    """Checks a 2-d operand and returns its row stride."""
    _need(t.dim() == 2, f"{name} must have two dimensions")
    _need(rows is None or t.shape[0] == rows, f"{name} must have {rows} rows, has {t.shape[0]}")
    _need(cols is None or t.shape[1] == cols, f"{name} must have {cols} columns, has {t.shape[1]}")
    r, c = t.shape
    _need(c <= 1 or t.stride(1) == 1, f"{name} must have unit column stride")
    if r <= 1:
        return c
    _need(t.stride(0) >= c, f"{name} must be row-major with rows that do not overlap")
    return t.stride(0)


def _stack(name: str, t: torch.Tensor) -> tuple[int, int]:
    """Checks a [experts, n, k] operand and returns its row and expert strides."""
    _need(t.dim() == 3, f"{name} must have three dimensions [experts, n, k]")
    e, n, k = t.shape
    _need(k <= 1 or t.stride(2) == 1, f"{name} must have unit stride in its last dimension")
    _need(n <= 1 or t.stride(1) >= k, f"{name}'s rows must not overlap")
    ld = t.stride(1) if n > 1 else k
    _need(e <= 1 or n == 0 or t.stride(0) >= (n - 1) * ld + k, f"{name}'s matrices must not overlap")
    return ld, t.stride(0) if e > 1 else n * ld


def _rows_apart(t: torch.Tensor) -> torch.Tensor:
    """A gradient as autograd hands it over may be a broadcast or transposed view."""
    r, c = t.shape[-2:]
    ok = (c <= 1 or t.stride(-1) == 1) and (r <= 1 or t.stride(-2) >= c)
    return t if ok else t.contiguous()


def _offsets(offsets: torch.Tensor, experts: int) -> None:
    _need(offsets.dtype == torch.int32 and offsets.dim() == 1 and offsets.is_contiguous()
          and offsets.shape[0] == experts + 1, f"offsets must be {experts + 1} contiguous 32-bit integers")


def _type(name: str, t: torch.Tensor, kinds) -> int:
    if t.dtype not in kinds:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}")
    return dtype_code(t.dtype)


def _out(out, rows, cols, dtype, device, inputs) -> tuple[torch.Tensor, bool]:
    """The output, and whether it is new (then the rows nobody computes are zeroed)."""
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), True
    _on_device(device, out=out)
    _need(out.dtype == dtype, f"out must be {dtype}")
    _matrix("out", out, rows, cols)
    _need(not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (*inputs, out))),
          "out= takes no part in autograd; call under torch.no_grad()")
    return out, False


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device: torch.device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


# ---------------------------------------------------------------------------- tokens by expert

@dataclass(frozen=True)
class TokenOrder:
    """A router's choices sorted by expert (made by ``sort_tokens``).

    offsets [num_experts + 1]: expert e owns sorted rows offsets[e] .. offsets[e + 1]; the last entry is
    the number of kept slots. slots [tokens * top_k]: sorted position to slot (token * top_k + j).
    rows [tokens, top_k]: slot to sorted position. All 32-bit.
    """
    offsets: torch.Tensor
    slots: torch.Tensor
    rows: torch.Tensor
    num_experts: int

    @property
    def tokens(self) -> int:
        return self.rows.shape[0]

    @property
    def top_k(self) -> int:
        return self.rows.shape[1]

    def kept_ptr(self) -> int:
        return self.offsets.data_ptr() + 4 * self.num_experts


def sort_tokens(experts: torch.Tensor, num_experts: int) -> TokenOrder:
    """Sort the slots of ``experts`` ([tokens, top_k] or [tokens] ids, 32- or 64-bit integers) by expert,
    slots of one expert in their own order. Ids outside [0, num_experts) are dropped: they sort behind
    the last expert. At most 1024 experts."""
    if experts.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"unsupported dtype {experts.dtype} of experts")
    _need(experts.is_cuda, "experts must be a device tensor")
    _need(experts.dim() in (1, 2), "experts must be [tokens, top_k] or [tokens]")
    num_experts = int(num_experts)
    ids = (experts if experts.dim() == 2 else experts[:, None]).contiguous()
    n, dev = ids.numel(), ids.device
    ws_bytes = _lib.experts_sort_workspace_bytes(n, num_experts)
    with torch.cuda.device(dev):
        offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
        slots = torch.empty(n, dtype=torch.int32, device=dev)
        rows = torch.empty(ids.shape, dtype=torch.int32, device=dev)
        ws = _workspace(ws_bytes, dev)
        _lib.experts_sort(ids.data_ptr(), 8 * ids.element_size(), n, num_experts, offsets.data_ptr(), slots.data_ptr(),
                          rows.data_ptr(), _ptr(ws), ws_bytes, _stream(dev))
    return TokenOrder(offsets, slots, rows, num_experts)


def _gather(x, order, out):
    code = _type("x", x, (*_16BIT, torch.float32))
    _on_device(x.device, x=x, rows=order.rows)
    ldx = _matrix("x", x, rows=order.tokens)
    out, fresh = _out(out, order.rows.numel(), x.shape[1], x.dtype, x.device, (x,))
    with torch.cuda.device(x.device):
        _lib.experts_gather(x.data_ptr(), code, order.tokens, order.top_k, x.shape[1], ldx, order.rows.data_ptr(),
                            order.kept_ptr(), out.data_ptr(), _matrix("out", out), fresh, _stream(x.device))
    return out


def _combine(y, order, weights, out):
    code = _type("y", y, (*_16BIT, torch.float32))
    _on_device(y.device, y=y, rows=order.rows, weights=weights)
    ldy = _matrix("y", y, rows=order.rows.numel())
    wcode = 0
    if weights is not None:
        wcode = _type("weights", weights, (*_16BIT, torch.float32))
        _need(tuple(weights.shape) == tuple(order.rows.shape), f"weights must be {tuple(order.rows.shape)}")
        weights = weights.contiguous()
    out, _ = _out(out, order.tokens, y.shape[1], y.dtype, y.device, (y, weights))
    with torch.cuda.device(y.device):
        _lib.experts_combine(y.data_ptr(), code, order.tokens, order.top_k, y.shape[1], ldy, order.rows.data_ptr(),
                             order.kept_ptr(), _ptr(weights), wcode, out.data_ptr(), _matrix("out", out),
                             _stream(y.device))
    return out


def gather_rows_grad(dsorted: torch.Tensor, order: TokenOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``gather_rows``: each token's sum over its kept rows of ``dsorted``, in fp32, rounded once."""
    return _combine(dsorted.detach(), order, None, out)


def combine_rows_grad(dout: torch.Tensor, y: torch.Tensor, order: TokenOrder,
                      weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradients of ``combine_rows`` for y and the weights (None without weights), in their types. Rows
    and weights of dropped slots get zeros."""
    code = _type("y", y, (*_16BIT, torch.float32))
    dev = y.device
    _on_device(dev, y=y, dout=dout, rows=order.rows, weights=weights)
    _need(dout.dtype == y.dtype, f"dout must be {y.dtype}")
    ldy = _matrix("y", y, rows=order.rows.numel())
    lddo = _matrix("dout", dout, rows=order.tokens, cols=y.shape[1])
    wcode, dw = 0, None
    if weights is not None:
        wcode = _type("weights", weights, (*_16BIT, torch.float32))
        _need(tuple(weights.shape) == tuple(order.rows.shape), f"weights must be {tuple(order.rows.shape)}")
        weights = weights.detach().contiguous()
        dw = torch.empty(order.rows.shape, dtype=weights.dtype, device=dev)
    dy = torch.empty(y.shape, dtype=y.dtype, device=dev)
    with torch.cuda.device(dev):
        _lib.experts_combine_grad(dout.data_ptr(), lddo, y.data_ptr(), code, order.tokens, order.top_k, y.shape[1], ldy,
                                  order.rows.data_ptr(), order.kept_ptr(), _ptr(weights), wcode, dy.data_ptr(),
                                  y.shape[1], _ptr(dw), True, _stream(dev))
    return dy, dw


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.order = order
        return _gather(x, order, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dsorted):
        return gather_rows_grad(_rows_apart(dsorted), ctx.order), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, order, weights):
        ctx.order = order
        ctx.save_for_backward(y, weights)
        return _combine(y, order, weights, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, weights = ctx.saved_tensors
        dy, dw = combine_rows_grad(_rows_apart(dout), y, ctx.order, weights)
        return dy, None, dw


def gather_rows(x: torch.Tensor, order: TokenOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows x [tokens, width] in the order's sorted rows [tokens * top_k, width]. Rows at dropped
    positions are zeros in a new tensor, and left as they were in ``out``."""
    return _Gather.apply(x, order) if out is None else _gather(x, order, out)


def combine_rows(y: torch.Tensor, order: TokenOrder, weights: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Each token's weighted sum of its kept sorted rows: y [tokens * top_k, width], weights [tokens,
    top_k] (fp32 or 16-bit; None: ones). Summed in fp32 in the slots' order, rounded once to y's type."""
    return _Combine.apply(y, order, weights) if out is None else _combine(y, order, weights, out)


# --------------------------------------------------------------------------- experts' products

def _grouped_run(mode, x, y, out, offsets, rows, experts, n, k, ldx, ldy, ldo, stride, fresh):
    p = _lib.GemmGrouped(mode=mode, rows=rows, experts=experts, n=n, k=k, in_dtype=dtype_code(x.dtype),
                         out_dtype=dtype_code(out.dtype), ldx=ldx, ldy=ldy, ldo=ldo, stride=stride, zero_rest=int(fresh))
    ws_bytes = _lib.gemm_grouped_workspace_bytes(p, x.data_ptr(), y.data_ptr())
    with torch.cuda.device(x.device):
        ws = _workspace(ws_bytes, x.device)
        _lib.gemm_grouped_run(p, x.data_ptr(), y.data_ptr(), out.data_ptr(), offsets.data_ptr(), _ptr(ws), ws_bytes,
                              _stream(x.device))
    return out


def _grouped_forward(A, B, offsets, out_dtype, out):
    _type("A", A, _16BIT)
    _need(B.dtype == A.dtype, f"B must be {A.dtype}")
    _on_device(A.device, A=A, B=B, offsets=offsets)
    ldb, stride = _stack("B", B)
    E, N, K = B.shape
    lda = _matrix("A", A, cols=K)
    _offsets(offsets, E)
    dtype = out.dtype if out is not None and out_dtype is None else out_dtype or A.dtype
    dtype_code(dtype)
    C, fresh = _out(out, A.shape[0], N, dtype, A.device, (A, B))
    return _grouped_run(_lib.GEMM_GROUPED_FORWARD, A, B, C, offsets, A.shape[0], E, N, K, lda, ldb, _matrix("out", C),
                        stride, fresh)


def grouped_matmul_grad_a(dC: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for A: dA[i] = dC[i]·B[e] for expert e's rows i, in dC's type. Rows behind
    the last expert: zeros in a new tensor, left as they were in ``out``."""
    dC, B = dC.detach(), B.detach()
    _type("dC", dC, _16BIT)
    _need(B.dtype == dC.dtype, f"B must be {dC.dtype}")
    _on_device(dC.device, dC=dC, B=B, offsets=offsets)
    ldb, stride = _stack("B", B)
    E, N, K = B.shape
    lddc = _matrix("dC", dC, cols=N)
    _offsets(offsets, E)
    dA, fresh = _out(out, dC.shape[0], K, dC.dtype, dC.device, ())
    return _grouped_run(_lib.GEMM_GROUPED_GRAD_A, dC, B, dA, offsets, dC.shape[0], E, N, K, lddc, ldb, _matrix("out", dA),
                        stride, fresh)


def grouped_matmul_grad_b(dC: torch.Tensor, A: torch.Tensor, offsets: torch.Tensor,
                          out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for B, [experts, n, k]: dB[e] = sum over expert e's rows i of
    dC[i]ᵀ·A[i], in A's type or ``out_dtype`` (fp32 for a main copy of the weights); zeros for an expert
    without rows."""
    dC, A = dC.detach(), A.detach()
    _type("A", A, _16BIT)
    _need(dC.dtype == A.dtype, f"dC must be {A.dtype}")
    _on_device(A.device, dC=dC, A=A, offsets=offsets)
    _need(offsets.dim() == 1 and offsets.shape[0] >= 1, "offsets must be [experts + 1]")
    E = offsets.shape[0] - 1
    _offsets(offsets, E)
    lddc = _matrix("dC", dC, rows=A.shape[0])
    lda = _matrix("A", A)
    N, K = dC.shape[1], A.shape[1]
    dtype = out_dtype or A.dtype
    dtype_code(dtype)
    dB = torch.empty((E, N, K), dtype=dtype, device=A.device)
    return _grouped_run(_lib.GEMM_GROUPED_GRAD_B, dC, A, dB, offsets, A.shape[0], E, N, K, lddc, lda, K, N * K, True)


class _Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B, offsets, out_dtype):
        ctx.save_for_backward(A, B, offsets)
        return _grouped_forward(A, B, offsets, out_dtype, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dC):
        A, B, offsets = ctx.saved_tensors
        dC = _rows_apart(dC.to(A.dtype))  # the products take 16-bit operands of one type
        dA = grouped_matmul_grad_a(dC, B, offsets) if ctx.needs_input_grad[0] else None
        dB = grouped_matmul_grad_b(dC, A, offsets) if ctx.needs_input_grad[1] else None
        return dA, dB, None, None


def grouped_matmul(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, out_dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """C[i] = A[i]·B[e]ᵀ for expert e's rows offsets[e] <= i < offsets[e + 1]: A [rows, k] and B [experts, n, k]
    fp16 or bf16, fp32 sums, C in A's type or ``out_dtype``. ``offsets``: 32-bit, on the device (a
    ``TokenOrder``'s). Rows behind the last expert are zeros in a new tensor, left as they were in ``out``."""
    if out is None:
        return _Grouped.apply(A, B, offsets, out_dtype)
    return _grouped_forward(A, B, offsets, out_dtype, out)


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


def pack_w4(q: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
            group_size: int = 128) -> W4Weight:
    """Lay out weights (q - z) * s: q [n, k] or [experts, n, k] bytes holding 0 .. 15 (the low four bits are
    taken), scales [..., n, ceil(k / group_size)] fp16 or bf16 (the products' type), zeros bytes of the same
    shape, or None for z = 8. group_size 32, 64 or 128."""
    _need(q.dtype == torch.uint8 and q.dim() in (2, 3), "q must be [n, k] or [experts, n, k] bytes")
    _type("scales", scales, _16BIT)
    _on_device(q.device, q=q, scales=scales, zeros=zeros)
    group_size = int(group_size)
    _need(group_size in (32, 64, 128), "group_size must be 32, 64 or 128")
    n, k = q.shape[-2:]
    shape = (*q.shape[:-1], -(-k // group_size))
    _need(tuple(scales.shape) == shape, f"scales must be {shape}")
    _need(zeros is None or (zeros.dtype == torch.uint8 and tuple(zeros.shape) == shape), f"zeros must be bytes {shape}")
    matrices = q.shape[0] if q.dim() == 3 else 1
    nbytes = _lib.gemm_w4_packed_bytes(matrices, n, k, group_size, zeros is not None)
    with torch.cuda.device(q.device):
        q, scales = q.contiguous(), scales.detach().contiguous()
        zeros = zeros.contiguous() if zeros is not None else None
        packed = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _lib.gemm_w4_pack(q.data_ptr(), scales.data_ptr(), _ptr(zeros), matrices, n, k, group_size, packed.data_ptr(),
                          _stream(q.device))
    return W4Weight(packed, matrices, q.dim() == 3, n, k, group_size, zeros is not None, scales.dtype)


def w4_matmul(x: torch.Tensor, w: W4Weight, offsets: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """x [rows, k] times the 4-bit weight, [rows, n]: one weight for all rows, or expert e's for rows
    offsets[e] <= i < offsets[e + 1] of a weight packed from [experts, n, k]. x in the scales' type; no weight
    is rounded, sums are fp32. No gradient. Rows behind the last expert are zeros in a new tensor, left as they
    were in ``out``."""
    _type("x", x, _16BIT)
    _need(x.dtype == w.dtype, f"x must be {w.dtype}, the scales' type")
    _on_device(x.device, x=x, weight=w.packed, offsets=offsets)
    _need((offsets is not None) == w.stacked,
          "offsets go with a weight packed from [experts, n, k], and only with one")
    _need(not (torch.is_grad_enabled() and x.requires_grad), "w4_matmul has no gradient; call under torch.no_grad()")
    ldx = _matrix("x", x, cols=w.k)
    if offsets is not None:
        _offsets(offsets, w.matrices)
    dtype = out.dtype if out is not None and out_dtype is None else out_dtype or x.dtype
    dtype_code(dtype)
    out, fresh = _out(out, x.shape[0], w.n, dtype, x.device, ())
    p = _lib.GemmW4(rows=x.shape[0], matrices=w.matrices, n=w.n, k=w.k, group=w.group_size,
                    has_zeros=int(w.has_zeros), dtype=dtype_code(x.dtype), out_dtype=dtype_code(dtype), ldx=ldx,
                    ldo=_matrix("out", out), zero_rest=int(fresh))
    with torch.cuda.device(x.device):
        ws_bytes = _lib.gemm_w4_workspace_bytes(p, offsets is not None)
        ws = _workspace(ws_bytes, x.device)
        _lib.gemm_w4_run(p, x.data_ptr(), w.packed.data_ptr(), _ptr(offsets), out.data_ptr(), _ptr(ws), ws_bytes,
                         _stream(x.device))
    return out


# --------------------------------------------------------------------------------- all together

def routed_matmul(x: torch.Tensor, weight: torch.Tensor | W4Weight, experts: torch.Tensor,
                  weights: torch.Tensor | None = None) -> torch.Tensor:
    """A routed linear layer: out[t] = sum over j of weights[t, j] * x[t]·B[experts[t, j]]ᵀ, with B
    [experts, n, k] 16-bit, or packed in 4 bits (no gradient then). The tokens are sorted by expert, their
    rows gathered, multiplied and combined; ids outside the experts are dropped. Differentiable in x, B and
    the weights."""
    four_bits = isinstance(weight, W4Weight)
    num = weight.matrices if four_bits else weight.shape[0]
    _need(not four_bits or weight.stacked, "the weight must be packed from [experts, n, k]")
    _need(experts.shape[0] == x.shape[0], f"experts must have {x.shape[0]} rows")
    order = sort_tokens(experts, num)
    rows = gather_rows(x, order)
    y = w4_matmul(rows, weight, order.offsets) if four_bits else grouped_matmul(rows, weight, order.offsets)
    if weights is not None and weights.dim() == 1:
        weights = weights[:, None]
    return combine_rows(y, order, weights)
