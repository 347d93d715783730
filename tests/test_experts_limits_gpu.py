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
