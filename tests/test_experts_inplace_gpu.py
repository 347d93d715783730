"""Tensors that autograd saved and that this package's calls, or their callers, write afterwards: backward has to
raise, as after torch's own writes, instead of computing with the new contents."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16 = torch.bfloat16


def ones(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype, device="cuda")


def calls():
    """name -> (a call that writes `out`, out's shape)"""
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [1, 1]], device="cuda")
    order = spt.sort_tokens(ids, 3)
    x, rows, b = ones(4, 32), ones(8, 32), ones(3, 32, 32)
    w = spt.pack_w4(torch.full((32, 32), 9, dtype=torch.uint8, device="cuda"), ones(32, 1), group_size=32)
    return {
        "gather_rows": (lambda out: spt.gather_rows(x, order, out=out), (8, 32)),
        "gather_rows_grad": (lambda out: spt.gather_rows_grad(rows, order, out=out), (4, 32)),
        "combine_rows": (lambda out: spt.combine_rows(rows, order, out=out), (4, 32)),
        "grouped_matmul": (lambda out: spt.grouped_matmul(rows, b, order.offsets, out=out), (8, 32)),
        "grouped_matmul_grad_a": (lambda out: spt.grouped_matmul_grad_a(rows, b, order.offsets, out=out), (8, 32)),
        "w4_matmul": (lambda out: spt.w4_matmul(x, w, out=out), (4, 32)),
    }


@pytest.mark.parametrize("name", ["gather_rows", "gather_rows_grad", "combine_rows", "grouped_matmul",
                                  "grouped_matmul_grad_a", "w4_matmul"])
@pytest.mark.parametrize("view", [False, True])
def test_writing_a_saved_out_is_seen(name, view):
    call, shape = calls()[name]
    buf = ones(shape[0] + 1, shape[1])
    out = buf[1:] if view else buf[1:].clone()
    saved = buf if view else out  # a view shares its base's version
    scale = torch.ones((), dtype=BF16, device="cuda", requires_grad=True)
    loss = (saved * scale).sum()
    with torch.no_grad():
        call(out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # a refused call has written nothing, and a new output touches no other tensor
    before = out._version
    with pytest.raises(ValueError):
        call(out[:-1])
    assert out._version == before


def test_a_gather_buffer_used_for_two_batches():
    # the second batch's rows must not stand in the first one's gradient
    order = spt.sort_tokens(torch.tensor([[0], [1], [1]], device="cuda"), 2)
    b = ones(2, 16, 16).requires_grad_()
    buf = ones(3, 16)
    spt.gather_rows(ones(3, 16), order, out=buf)
    first = spt.grouped_matmul(buf, b, order.offsets)
    spt.gather_rows(2 * ones(3, 16), order, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        first.sum().backward()


@pytest.mark.parametrize("through", ["matmul", "plan"])
def test_the_dense_product_writing_a_saved_out_is_seen(through):
    a, b, buf = ones(4, 32), ones(16, 32), ones(4, 16)
    experts = ones(1, 8, 16).requires_grad_()
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    first = spt.grouped_matmul(buf, experts, off)
    if through == "matmul":
        spt.matmul(a, b, out=buf)
    else:
        spt.Plan(4, 16, 32, BF16, BF16).run(a, b, buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        first.sum().backward()
    assert torch.equal(spt.matmul(a, b), buf)


def test_out_made_in_inference_mode():
    with torch.inference_mode():
        order = spt.sort_tokens(torch.tensor([[0], [1]], device="cuda"), 2)
        x = ones(2, 16)
        assert torch.equal(spt.gather_rows(x, order, out=torch.empty_like(x)), x)
