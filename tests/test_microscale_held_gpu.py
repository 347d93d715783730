"""GPU tests of microscaled tensors moved between host and device."""
import pickle

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402


@pytest.mark.parametrize("bits", [4, 8])
def test_there_and_back(bits, tmp_path):
    x = torch.randn((70, 300), device="cuda", dtype=torch.bfloat16)
    w = spt.quantize_mx(torch.randn((90, 300), device="cuda"), 4)
    q = spt.quantize_mx(x, bits)
    want, product = spt.dequantize_mx(q), spt.mx_matmul(q, w)
    assert q.to("cuda") is q and q.to(q.device) is q
    torch.save(q, tmp_path / "q.pt")
    loaded = torch.load(tmp_path / "q.pt", map_location="cpu", weights_only=False)  # written above
    for held in (q.to("cpu"), loaded, pickle.loads(pickle.dumps(q.to("cpu")))):
        assert held.device.type == "cpu" and torch.equal(held.codes, q.codes.cpu()) and torch.equal(held.scales, q.scales.cpu())
        with pytest.raises(ValueError, match="device tensor"):
            spt.dequantize_mx(held)
        with pytest.raises(ValueError, match="on cpu|device tensor"):
            spt.mx_matmul(q, held) if bits == 4 else spt.mx_matmul(held, w)
        back = held.to("cuda")
        assert back.codes_ptr != q.codes_ptr and back.dtype == q.dtype
        assert torch.equal(spt.dequantize_mx(back), want) and torch.equal(spt.mx_matmul(back, w), product)
