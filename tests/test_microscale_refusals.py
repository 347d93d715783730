"""What the microscaled calls refuse rather than answer wrongly, on a host without a GPU."""
import pytest
import torch
from torch.autograd import forward_ad

import software_pipelined_tiled_amd as spt

C8, S8 = torch.zeros(4, 40).to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8)


def test_codes_in_a_graph():
    """8-bit codes may be a type that takes part in autograd; the layout does not."""
    leaf = torch.zeros(4, 40).to(torch.float8_e4m3fn).requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_mx(leaf, S8, 8)
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_mx(torch.zeros(4, 40, requires_grad=True).to(torch.float8_e4m3fn), S8, 8)
    for call in (lambda: spt.pack_mx(C8, S8, 8), lambda: spt.pack_mx(leaf.detach(), S8, 8)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
        spt.pack_mx(leaf, S8, 8)


def test_scales_in_a_graph():
    scales = torch.ones(4, 2).to(torch.float8_e8m0fnu).requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_mx(C8, scales, 8)


def test_codes_with_a_tangent():
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(C8, C8.clone())
        with pytest.raises(ValueError, match="forward-mode"):
            spt.pack_mx(dual, S8, 8)
