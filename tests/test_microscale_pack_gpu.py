"""GPU tests of the layout where a row's last group of 512 columns is whole, and of the rows and columns beside that."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402
from test_microscale_gpu import codes_of, gen, plain_codes, scale_bytes  # noqa: E402


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows", [15, 16, 17, 64, 100])
@pytest.mark.parametrize("k", [511, 512, 513, 544, 1023, 1024, 2048, 2049])
def test_whole_groups(rows, k, bits):
    """Rows at odd distances and begins, with other bytes all around: every code and scale, zeros behind them, nothing else."""
    g = gen(rows + k)
    codes = torch.randint(0, 16 if bits == 4 else 256, (rows, k), generator=g, device="cuda")
    scales = torch.randint(0, 256, (rows, -(-k // 32)), generator=g, device="cuda").to(torch.uint8)
    plain = plain_codes(codes, bits, k)
    for before, behind in ((0, 0), (0, 1), (1, 0), (3, 4), (5, 8)):
        c = torch.full((rows, before + plain.shape[1] + behind), 255, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, before + scales.shape[1] + behind), 255, dtype=torch.uint8, device="cuda")
        cv, sv = c[:, before:before + plain.shape[1]], s[:, before:before + scales.shape[1]]
        cv.copy_(plain)
        sv.copy_(scales)
        q = spt.pack_mx(cv, sv, bits, k)
        assert torch.equal(codes_of(q)[:, :k], codes) and not codes_of(q)[:, k:].any()
        assert torch.equal(scale_bytes(q)[:, : sv.shape[1]], scales) and not scale_bytes(q)[:, sv.shape[1]:].any()
        if rows % 64:
            assert not q.scales[-1, :, rows % 64:].any()
