"""Sizes near the limits of the experts' operators and 4-bit products, on the device."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16 = torch.bfloat16


def ints(shape, seed, top=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("matrices", [0, 5])
def test_4_bit_products_of_more_rows_than_16_row_blocks(matrices):
    # few columns and a long sum: kernels of 16 rows a block are the fastest, and have too many blocks
    rows, n, k, group = 65535 * 16 + 1, 16, 1024, 128
    shape = (matrices, n) if matrices else (n,)
    q = torch.randint(0, 16, (*shape, k), device="cuda", dtype=torch.uint8)
    w = spt.pack_w4(q, torch.ones((*shape, k // group), dtype=BF16, device="cuda"), group_size=group)
    dense = q.to(torch.float64) - 8
    x = ints((rows, k), 1)
    bounds = [0, 3, 3, 500_000, 1_000_000, rows] if matrices else [0, rows]
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda") if matrices else None
    got = spt.w4_matmul(x, w, off, out_dtype=torch.float32)
    for at in (0, 2, 3, 499_999, 500_000, 524_287, 999_999, 1_000_000, rows - 2, rows - 1):
        e = max(i for i in range(len(bounds) - 1) if bounds[i] <= at < bounds[i + 1])
        want = x[at].to(torch.float64) @ (dense[e] if matrices else dense).t()
        assert torch.equal(got[at].to(torch.float64), want), at
    # every row: the sum over columns equals the product with the summed columns (whole numbers, exact)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        col = (dense[e] if matrices else dense).sum(0, keepdim=True)
        for i in range(lo, hi, 1 << 17):
            j = min(hi, i + (1 << 17))
            assert torch.equal(got[i:j].to(torch.float64).sum(1, keepdim=True), x[i:j].to(torch.float64) @ col.t())


@pytest.mark.parametrize("tile", [32, 128, 256])
@pytest.mark.parametrize("grad", [False, True])
def test_experts_that_claim_the_same_rows_add_no_work(tile, grad):
    # wrong contents of offsets: four experts have all rows each. The walk over the output tiles ends with the most
    # tiles that ascending offsets can have, so the last experts' are not computed, and nothing outside is touched.
    rows, k, n = 8 * tile, 32, 48
    x = torch.ones((rows, n if grad else k), dtype=BF16, device="cuda")
    # experts 0, 2, 4 and 6 have the rows, with weights 1, 2, 3 and 4; those between have none
    b = torch.tensor([1, 0, 2, 0, 3, 0, 4], dtype=BF16, device="cuda")[:, None, None].repeat(1, n, k)
    off = torch.tensor([0, rows, 0, rows, 0, rows, 0, rows], dtype=torch.int32, device="cuda")
    out = torch.full((rows + 128, k if grad else n), 7.0, dtype=BF16, device="cuda")
    (spt.grouped_matmul_grad_a if grad else spt.grouped_matmul)(x, b, off, out=out[64:-64], tile=tile)
    length = n if grad else k
    assert ((out[64:-64] == length) | (out[64:-64] == 2 * length)).all()
    assert (out[:64] == 7).all() and (out[-64:] == 7).all()
