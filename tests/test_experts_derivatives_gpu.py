"""Derivatives of the experts' operators: an order changed before backward is seen, and derivatives that the operators
do not have (of a gradient, of the scales, in forward mode) are refused, not left out."""
import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16 = torch.bfloat16


def ones(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype, device="cuda")


def operands():
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [1, 1]], device="cuda")
    return ids, spt.sort_tokens(ids, 3), ones(4, 32), ones(8, 32), ones(3, 32, 32), ones(4, 2)


# ------------------------------------------------------------------------------- the saved order

@pytest.mark.parametrize("name", ["gather_rows", "combine_rows"])
@pytest.mark.parametrize("part", ["rows", "offsets"])
def test_an_order_changed_before_backward_is_seen(name, part):
    _, order, x, rows, _, w = operands()
    if name == "gather_rows":
        out = spt.gather_rows(x.requires_grad_(), order)
    else:
        out = spt.combine_rows(rows.requires_grad_(), order, w)
    getattr(order, part).add_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_saved_orders_through_hooks():
    # tensors saved for backward may come back as copies
    ids, _, x, _, b, w = operands()
    leaves = [t.clone().requires_grad_() for t in (x, b, w)]

    def train():
        return torch.autograd.grad(spt.routed_matmul(leaves[0], leaves[1], ids, leaves[2]).float().square().sum(), leaves)
    want = train()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.cpu(), lambda t: t.cuda()):
        got = train()
    for g, e in zip(got, want):
        assert torch.equal(g, e)


@pytest.mark.parametrize("wanted", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_gradients_of_some_inputs_only(wanted):
    ids, _, x, _, b, w = operands()
    def grads(which):
        leaves = [t.clone().requires_grad_(on) for t, on in zip((x, b, w), which)]
        spt.routed_matmul(leaves[0], leaves[1], ids, leaves[2]).float().square().sum().backward()
        return [t.grad for t in leaves]
    for got, want, on in zip(grads(wanted), grads((True, True, True)), wanted):
        assert torch.equal(got, want) if on else got is None


# ---------------------------------------------------------------------- derivatives of the gradients

def gradient_calls():
    """name -> (the call on its tensors, the tensors)"""
    _, order, x, rows, b, w = operands()
    off = order.offsets
    return {
        "gather_rows_grad": (lambda d: spt.gather_rows_grad(d, order), [rows]),
        "combine_rows_grad": (lambda d, y, w: spt.combine_rows_grad(d, y, order, w), [x, rows, w]),
        "combine_rows_grad without weights": (lambda d, y: spt.combine_rows_grad(d, y, order)[0], [x, rows]),
        "grouped_matmul_grad_a": (lambda d, b: spt.grouped_matmul_grad_a(d, b, off), [rows, b]),
        "grouped_matmul_grad_b": (lambda d, a: spt.grouped_matmul_grad_b(d, a, off, torch.float32), [rows, rows.clone()]),
    }


@pytest.mark.parametrize("name,which", [("gather_rows_grad", 0), ("combine_rows_grad", 0), ("combine_rows_grad", 1),
                                        ("combine_rows_grad", 2), ("combine_rows_grad without weights", 0),
                                        ("grouped_matmul_grad_a", 0), ("grouped_matmul_grad_a", 1),
                                        ("grouped_matmul_grad_b", 0), ("grouped_matmul_grad_b", 1)])
def test_a_gradient_of_a_gradient_raises(name, which):
    call, args = gradient_calls()[name]
    def each(r):
        return r if isinstance(r, tuple) else (r,)
    want = each(call(*args))
    leaf = args[which].clone().requires_grad_()
    args[which] = leaf
    got = each(call(*args))
    for g, e in zip(got, want):
        assert torch.equal(g, e)
        # beside a term that has its derivative, so that a lost one would not be noticed
        with pytest.raises(RuntimeError, match="differentiable once"):
            (leaf.float().sum() + g.float().square().sum()).backward()
    with torch.no_grad():
        assert not any(g.requires_grad for g in each(call(*args)))


def test_out_takes_no_part_in_a_graph():
    _, order, _, rows, b, _ = operands()
    leaf = rows.clone().requires_grad_()
    for call in (lambda: spt.gather_rows_grad(leaf, order, out=ones(4, 32)),
                 lambda: spt.gather_rows_grad(rows, order, out=ones(4, 32).requires_grad_()),
                 lambda: spt.grouped_matmul_grad_a(leaf, b, order.offsets, out=ones(8, 32)),
                 lambda: spt.grouped_matmul_grad_a(rows, b.clone().requires_grad_(), order.offsets, out=ones(8, 32))):
        with pytest.raises(ValueError, match="no part in autograd"):
            call()
        with torch.no_grad():
            call()


# ---------------------------------------------------------------------------------- the scales

def test_scales_that_require_grad_are_refused():
    q = torch.full((32, 32), 9, dtype=torch.uint8, device="cuda")
    s = ones(32, 1).requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_w4(q, s, group_size=32)
    with torch.no_grad():
        w = spt.pack_w4(q, s, group_size=32)
    assert torch.equal(spt.w4_matmul(ones(4, 32), w), 32 * ones(4, 32))


# ---------------------------------------------------------------------------------- forward mode

def test_tensors_with_a_tangent_are_refused():
    ids, order, x, rows, b, w = operands()
    off = order.offsets
    q = torch.full((32, 32), 9, dtype=torch.uint8, device="cuda")
    w4 = spt.pack_w4(q, ones(32, 1), group_size=32)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        bad = [
            lambda: spt.gather_rows(dual(x), order), lambda: spt.gather_rows(dual(x), order, out=rows.clone()),
            lambda: spt.gather_rows(x, order, out=dual(rows.clone())),
            lambda: spt.combine_rows(dual(rows), order), lambda: spt.combine_rows(rows, order, dual(w)),
            lambda: spt.grouped_matmul(dual(rows), b, off), lambda: spt.grouped_matmul(rows, dual(b), off),
            lambda: spt.w4_matmul(dual(x), w4), lambda: spt.w4_matmul(x, w4, out=dual(x.clone())),
            lambda: spt.pack_w4(q, dual(ones(32, 1)), group_size=32),
            lambda: spt.gather_rows_grad(dual(rows), order), lambda: spt.gather_rows_grad(rows, order, out=dual(x.clone())),
            lambda: spt.combine_rows_grad(dual(x), rows, order), lambda: spt.combine_rows_grad(x, dual(rows), order),
            lambda: spt.combine_rows_grad(x, rows, order, dual(w)),
            lambda: spt.grouped_matmul_grad_a(dual(rows), b, off), lambda: spt.grouped_matmul_grad_a(rows, dual(b), off),
            lambda: spt.grouped_matmul_grad_b(dual(rows), rows, off), lambda: spt.grouped_matmul_grad_b(rows, dual(rows), off),
            lambda: spt.routed_matmul(dual(x), b, ids, w), lambda: spt.routed_matmul(x, dual(b), ids, w),
            lambda: spt.routed_matmul(x, b, ids, dual(w)),
            lambda: spt.gather_rows(dual(x.clone().requires_grad_()), order),
        ]
        for i, call in enumerate(bad):
            for mode in (torch.no_grad, torch.enable_grad):
                with mode(), pytest.raises(ValueError, match="forward-mode"):
                    call()
                    print("not refused:", i)
        # tensors without a tangent pass inside a level, and so does a backward of them
        leaf = x.clone().requires_grad_()
        spt.routed_matmul(leaf, b, ids, w).sum().backward()
        assert leaf.grad is not None
        # a gradient that arrives with a tangent
        out = spt.gather_rows(leaf, order)
        with pytest.raises(ValueError, match="forward-mode"):
            torch.autograd.grad(out, leaf, dual(torch.ones_like(out)))
    assert torch.equal(spt.gather_rows(x, order), rows)


# -------------------------------------------------------------------------------------- captured

@pytest.mark.parametrize("grad_mode", [False, True])
def test_gradients_of_leaves_captured_while_eager_ones_live(grad_mode):
    # a training step by the gradients' own calls, with parameters as operands: its results stay in the graph where
    # grad mode is on, and neither they nor eager results of the same leaves stand in the way of a capture
    _, order, _, rows, b, _ = operands()
    b.requires_grad_()
    dc = torch.arange(8, device="cuda", dtype=BF16)[:, None].repeat(1, 32)

    def step():
        da = spt.grouped_matmul_grad_a(dc, b, order.offsets)
        return [da, spt.grouped_matmul_grad_b(dc, rows, order.offsets), spt.gather_rows_grad(da, order)]
    with torch.set_grad_enabled(grad_mode):
        eager = step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
    for rep in range(3):
        dc.add_(1)
        g.replay()
        with torch.no_grad():
            want = step()
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            assert torch.equal(a, e), rep
    assert eager[0].requires_grad == grad_mode and got[0].requires_grad == grad_mode
