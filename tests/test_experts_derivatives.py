"""Derivatives that the experts' operators refuse before any device work."""
import pytest
import torch
from torch.autograd import forward_ad

import software_pipelined_tiled_amd as spt


def test_scales_that_require_grad():
    q, s = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_w4(q, s, group_size=32)
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
        spt.pack_w4(q, s, group_size=32)


def test_tensors_with_a_tangent():
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    order, off, b = spt.TokenOrder(i32(3), i32(4), i32(4, 1), 2), i32(3), torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    calls = [lambda d: spt.gather_rows(d, order), lambda d: spt.combine_rows(d, order), lambda d: spt.gather_rows_grad(d, order),
             lambda d: spt.combine_rows_grad(t, d, order), lambda d: spt.grouped_matmul(d, b, off),
             lambda d: spt.grouped_matmul_grad_a(d, b, off), lambda d: spt.grouped_matmul_grad_b(t, d, off),
             lambda d: spt.pack_w4(torch.zeros((4, 256), dtype=torch.uint8), d, group_size=32)]
    for call in calls:
        with forward_ad.dual_level(), torch.no_grad():
            with pytest.raises(ValueError, match="forward-mode"):
                call(forward_ad.make_dual(t, torch.ones_like(t)))
            with pytest.raises(ValueError, match="device tensor"):
                call(t)
        with pytest.raises(ValueError, match="device tensor"):
            call(t)
