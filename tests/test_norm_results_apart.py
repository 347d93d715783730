"""The norm writes two results, h and y: calls that give both the same memory are refused, in C and from Python."""
import ctypes

import pytest
import torch

import software_pipelined_tiled_amd as spt
from software_pipelined_tiled_amd import _lib

ROWS, N = 4, 40
BASE = 0x100000  # an address that no refused call reads
TYPES = [(spt.GEMM_BF16, 2), (spt.GEMM_F16, 2), (spt.GEMM_F32, 4)]


def run(dtype, y, ldy, h, ldh, rows=ROWS):
    p = _lib.NormRms(rows, N, dtype, spt.GEMM_F32, 1e-6, N, N, ldh, ldy)
    return spt.lib().norm_rms_run(ctypes.byref(p), BASE << 8, BASE << 9, None, h, y, None)


def share(y, ldy, h, ldh, rows=ROWS):
    """By the elements themselves."""
    cells = lambda at, ld: {at + r * ld + c for r in range(rows) for c in range(N)}  # noqa: E731
    return bool(cells(y, ldy) & cells(h, ldh))


@pytest.mark.parametrize("dtype,es", TYPES)
@pytest.mark.parametrize("ld", [40, 41, 79, 80, 100])
def test_rows_of_one_stride(dtype, es, ld):
    """Refused where an element is in both, and nowhere else. What is not refused goes on to the device: left to hosts without one."""
    for rows in (1, ROWS):
        for apart in range(0, ROWS * ld + 2 * N):
            for y, h in ((0, apart), (apart, 0)):
                if share(y, ld, h, ld, rows):
                    assert run(dtype, BASE + y * es, ld, BASE + h * es, ld, rows) == _lib.GEMM_ERR_INVALID, (rows, y, h)
                elif not torch.cuda.is_available():
                    assert run(dtype, BASE + y * es, ld, BASE + h * es, ld, rows) == _lib.GEMM_ERR_HIP, (rows, y, h)


def test_one_address_and_two_strides():
    for dtype, _ in TYPES:
        assert run(dtype, BASE, 40, BASE, 60) == _lib.GEMM_ERR_INVALID


@pytest.mark.parametrize("bits", [4, 8])
def test_microscaled_result(bits):
    p = _lib.NormRms(ROWS, N, spt.GEMM_BF16, spt.GEMM_F32, 1e-6, N, N, N, 0)
    for codes, scales in ((BASE, BASE << 1), (BASE << 1, BASE)):
        assert spt.lib().norm_rms_mx_run(ctypes.byref(p), bits, BASE << 8, BASE << 9, None, BASE, codes, scales, None) == _lib.GEMM_ERR_INVALID


def test_from_python():
    x, r = torch.zeros(ROWS, N, dtype=torch.bfloat16), torch.zeros(ROWS, N, dtype=torch.bfloat16)
    for both in (x, r, torch.zeros_like(x)):
        with pytest.raises(ValueError, match="memory of their own"):
            spt.rms_norm(x, residual=r, out=both, residual_out=both)
    with pytest.raises(ValueError, match="memory of their own"):
        spt.rms_norm(x, residual=r, out=x, residual_out=x.view(ROWS, N))
    with pytest.raises(ValueError, match="device tensor"):
        spt.rms_norm(x, residual=r, out=x, residual_out=r)
