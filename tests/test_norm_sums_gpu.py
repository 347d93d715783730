"""GPU tests of the norm's sums over a row, against what their order may lose."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BIG = 2.0**24


@pytest.mark.parametrize("waves,n", [(16, 8192), (8, 4096), (4, 2048), (2, 1024)])
@pytest.mark.parametrize("first,last", [(0, -1), (-1, 0), (0, 1), (1, 2)])
def test_waves_sums_meet_in_pairs(waves, n, first, last):
    """sum(g h) of one 2^24, one -2^24 and ones, each in a wave of its own (512 columns). In pairs only the two partial sums with the large
    values round, by at most 1 at each level until they meet: 2 (log2(waves) - 1). One after the other every 1 between them is lost."""
    first, last = first % waves, last % waves
    if first == last:
        return
    h = torch.ones((1, n), device="cuda")
    dy = torch.zeros((1, n), device="cuda")
    ones = 0
    for w in range(waves):
        at = 512 * w + 64 * (w % 8)  # another lane in each
        dy[0, at] = BIG if w == first else -BIG if w == last else 1.0
        ones += w not in (first, last)
    dx, _ = spt.rms_norm_grad(dy, h, None, eps=0.0)  # r = 1: dx = dy - sum(g h) / n
    free = dy[0] == 0
    got = -dx[0, free].double() * n
    assert (got == got[0]).all()
    assert abs(got[0].item() - ones) <= 2 * (waves.bit_length() - 2), (got[0].item(), ones)


@pytest.mark.parametrize("n", [1024, 1536, 4096, 4608, 8192, 16384])
def test_every_wave_counts(n):
    """Integers: the sums are exact in any order, whatever the number of waves; each place of the row once by itself."""
    dy = torch.zeros((n // 64, n), device="cuda")
    at = torch.arange(n // 64, device="cuda") * 64 + torch.arange(n // 64, device="cuda") % 64
    dy[torch.arange(n // 64, device="cuda"), at] = 1024.0
    h = torch.ones((n // 64, n), device="cuda")
    dx, _ = spt.rms_norm_grad(dy, h, None, eps=0.0)
    want = dy.double() - 1024.0 / n
    # r is off by v through 1 / n where n is no power of two, by as much again in the root and the division, and each product by v / 2
    assert ((dx.double() - want).abs() <= 16 * 2.0**-24 * (dy.double() + 1024.0 / n)).all()
