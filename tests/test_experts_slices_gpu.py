"""Some experts of an order: offsets[lo : hi + 1] with the weights of experts lo .. hi - 1. The rows in front of the
first expert belong to nobody, as those behind the last: zeros in a new tensor, left as they were in `out`."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def ints(shape, seed, top=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(BF16)


def stale(shape, dtype):
    """Leaves a block of NaN of this size with torch's allocator, for the next new tensor to land on."""
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# rows of each expert, then the experts taken
COUNTS = [([3, 70, 0, 129, 5], 1, 4), ([3, 70, 0, 129, 5], 4, 5), ([0, 0, 40, 1], 2, 3), ([7, 9], 1, 1), ([1, 1, 1], 2, 3),
          ([300, 257, 2], 1, 3), ([5] * 70, 3, 69), ([5] * 70, 66, 70), ([2, 0, 1, 1], 2, 4), ([600, 3], 2, 2)]


def bounds_of(counts, lo, hi, behind):
    off = torch.tensor([0, *np.cumsum(counts).tolist()], dtype=torch.int32, device="cuda")
    return off[lo:hi + 1], int(off[lo]), int(off[hi]), int(off[-1]) + behind


@pytest.mark.parametrize("counts,lo,hi", COUNTS)
@pytest.mark.parametrize("n,k", [(72, 88), (130, 2100), (2100, 130), (33, 45)])
@pytest.mark.parametrize("mode", ["f", "a"])
@pytest.mark.parametrize("behind", [0, 4])
def test_grouped_products(counts, lo, hi, n, k, mode, behind):
    off, first, last, rows = bounds_of(counts, lo, hi, behind)
    b = ints((hi - lo, n, k), 1)
    width, cols = (k, n) if mode == "f" else (n, k)
    x = ints((rows, width), 2)
    ref = torch.zeros((rows, cols), dtype=F64, device="cuda")
    for e in range(hi - lo):
        s = slice(int(off[e]), int(off[e + 1]))
        ref[s] = x[s].to(F64) @ (b[e].to(F64).t() if mode == "f" else b[e].to(F64))
    x[:first], x[last:] = float("nan"), float("inf")
    fn = spt.grouped_matmul if mode == "f" else spt.grouped_matmul_grad_a
    for tile in (0, 32, 128, 256):
        stale((rows, cols), BF16)
        assert torch.equal(fn(x, b, off, tile=tile), ref.to(BF16)), tile
        out = torch.full((rows, cols + 3), 7.0, dtype=BF16, device="cuda")
        fn(x, b, off, out=out[:, :cols], tile=tile)
        assert torch.equal(out[first:last, :cols], ref[first:last].to(BF16)), tile
        assert (out[:first] == 7).all() and (out[last:] == 7).all() and (out[:, cols:] == 7).all(), tile


@pytest.mark.parametrize("counts,lo,hi", COUNTS)
@pytest.mark.parametrize("tile", [0, 128, 256])
def test_gradient_of_the_weights(counts, lo, hi, tile):
    off, first, last, rows = bounds_of(counts, lo, hi, 3)
    dc, a = ints((rows, 72), 3), ints((rows, 88), 4)
    ref = torch.stack([dc[off[e]:off[e + 1]].to(F64).t() @ a[off[e]:off[e + 1]].to(F64) for e in range(hi - lo)]) if hi > lo \
        else torch.zeros((0, 72, 88), dtype=F64, device="cuda")
    dc[:first], a[:first], dc[last:], a[last:] = (float("nan"),) * 4
    assert torch.equal(spt.grouped_matmul_grad_b(dc, a, off, out_dtype=F32, tile=tile).to(F64), ref)


@pytest.mark.parametrize("counts,lo,hi", COUNTS)
@pytest.mark.parametrize("n,k", [(16, 4096), (72, 160), (1030, 512)])
def test_4_bit_experts(counts, lo, hi, n, k):
    off, first, last, rows = bounds_of(counts, lo, hi, 2)
    q = torch.randint(0, 16, (hi - lo, n, k), device="cuda", dtype=torch.uint8)
    w = spt.pack_w4(q, torch.ones((hi - lo, n, -(-k // 32)), dtype=BF16, device="cuda"), group_size=32)
    x = ints((rows, k), 5, 1)
    ref = torch.zeros((rows, n), dtype=F64, device="cuda")
    for e in range(hi - lo):
        s = slice(int(off[e]), int(off[e + 1]))
        ref[s] = x[s].to(F64) @ (q[e].to(F64) - 8).t()
    x[:first], x[last:] = float("nan"), float("inf")
    stale((rows, n), F32)
    assert torch.equal(spt.w4_matmul(x, w, off, out_dtype=F32).to(F64), ref)
    out = torch.full((rows, n + 1), 7.0, dtype=F32, device="cuda")
    spt.w4_matmul(x, w, off, out=out[:, :n])
    assert torch.equal(out[first:last, :n].to(F64), ref[first:last])
    assert (out[:first] == 7).all() and (out[last:] == 7).all() and (out[:, n] == 7).all()


def test_two_halves_of_the_experts_make_the_whole_layer():
    # as two devices that hold half of the experts each would, and the gradients of it
    tokens, n, k = 50, 40, 48
    ids = torch.randint(0, 6, (tokens, 2), device="cuda")
    order = spt.sort_tokens(ids, 6)
    w = torch.rand((tokens, 2), device="cuda")
    dout = ints((tokens, n), 6)

    def layer(parts):
        x, b = ints((tokens, k), 7).requires_grad_(), ints((6, n, k), 8).requires_grad_()
        rows = spt.gather_rows(x, order)
        y = 0
        for lo, hi in parts:
            stale((2 * tokens, n), BF16)
            y = y + spt.grouped_matmul(rows, b[lo:hi], order.offsets[lo:hi + 1])
        return torch.autograd.grad(spt.combine_rows(y, order, w), (x, b), dout)
    for got, want in zip(layer([(0, 2), (2, 6)]), layer([(0, 6)])):
        assert torch.equal(got, want)
