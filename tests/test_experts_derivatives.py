"""Derivatives that the experts' operators refuse before any device work."""
import pytest
import torch

import software_pipelined_tiled_amd as spt


def test_scales_that_require_grad():
    q, s = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="no gradient"):
        spt.pack_w4(q, s, group_size=32)
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
        spt.pack_w4(q, s, group_size=32)
