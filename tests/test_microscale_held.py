"""Microscaled tensors in host memory: they are loaded, copied and moved; every call on them is refused before it reads them."""
import copy
import pickle

import pytest
import torch

import software_pipelined_tiled_amd as spt
from software_pipelined_tiled_amd.microscale import MXTensor


def on_host(rows=70, k=300, bits=8, dtype=torch.bfloat16):
    """As a pickle written on a GPU comes back where there is none: two views of one storage."""
    blocks = -(-k // 128) * 4
    codes, scales = rows * blocks * 4 * bits, -(-rows // 64) * blocks * 64
    data = torch.arange(codes + scales, dtype=torch.int64).to(torch.uint8)
    call, args = MXTensor.__reduce__(_Parts(data[:codes].view(rows, blocks * 4 * bits), data[codes:].view(-(-rows // 64), blocks, 64), bits, rows, k, dtype))
    return call(*args)


class _Parts:
    def __init__(self, codes, scales, bits, rows, k, dtype):
        self.codes, self.scales, self.bits, self.rows, self.k, self.dtype = codes, scales, bits, rows, k, dtype


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,k", [(70, 300), (1, 1), (64, 128), (0, 5), (5, 0)])
def test_loaded_and_copied(rows, k, bits):
    q = on_host(rows, k, bits)
    assert q.shape == (rows, k) and q.device.type == "cpu" and q.to("cpu") is q
    for other in (copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
        assert torch.equal(other.codes, q.codes) and torch.equal(other.scales, q.scales)
        assert (other.bits, other.shape, other.dtype) == (q.bits, q.shape, q.dtype)
        assert other.codes_ptr == other.codes.data_ptr() and other.scales_ptr == other.scales.data_ptr()
    if rows and k:
        assert copy.deepcopy(q).codes_ptr != q.codes_ptr and copy.copy(q).codes_ptr == q.codes_ptr


def test_a_pickle_off_16_bytes():
    """Where the bytes lie in a file's mapping is not the tensor's doing; on a GPU they get memory of their own."""
    data = torch.zeros(70 * 384 + 2 * 12 * 64 + 8, dtype=torch.uint8)[8:]
    call, args = MXTensor.__reduce__(_Parts(data[: 70 * 384].view(70, 384), data[70 * 384:].view(2, 12, 64), 8, 70, 300, torch.float16))
    assert call(*args).codes.data_ptr() % 16 == 8


@pytest.mark.parametrize("change", [dict(bits=4), dict(rows=60), dict(k=400), dict(dtype=torch.float64)])
def test_parts_that_do_not_fit(change):
    q = on_host()
    parts = dict(codes=q.codes, scales=q.scales, bits=8, rows=70, k=300, dtype=torch.bfloat16)
    parts.update(change)
    call, args = MXTensor.__reduce__(_Parts(**parts))
    with pytest.raises((ValueError, TypeError)):
        call(*args)


def test_calls_are_refused():
    q, w = on_host(), on_host(40, 300, 4)
    x = torch.zeros(3, 300)
    for call in (lambda: spt.dequantize_mx(q), lambda: spt.dequantize_mx(q, out=torch.zeros(70, 300, dtype=torch.bfloat16)),
                 lambda: spt.mx_matmul(q, w), lambda: spt.mx_matmul(q, q, torch.float32), lambda: spt.mx_linear(x, w),
                 lambda: MXTensor(q.codes, q.scales, 8, 70, 300, torch.bfloat16)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
