"""Where the experts' operators and 4-bit products refuse a size, on the host."""
import ctypes

import pytest

import software_pipelined_tiled_amd as spt
from software_pipelined_tiled_amd import _lib

OK, INVALID, UNSUPPORTED = _lib.GEMM_OK, _lib.GEMM_ERR_INVALID, _lib.GEMM_ERR_UNSUPPORTED
BF16 = spt.GEMM_BF16


def w4_status(rows, n, k, matrices=1, offsets=False):
    p = _lib.GemmW4(rows=rows, matrices=matrices, n=n, k=k, group=128, has_zeros=0, dtype=BF16, out_dtype=BF16, ldx=k, ldo=n)
    return spt.lib().gemm_w4_workspace_bytes(ctypes.byref(p), int(offsets), ctypes.byref(ctypes.c_int64()))


# The limit is 65535 blocks of 64 rows, whichever kernel would be fastest for the size
@pytest.mark.parametrize("n", [16, 32, 64, 4096])
@pytest.mark.parametrize("k", [128, 1024, 4096, 8192])
@pytest.mark.parametrize("rows,status", [(65535 * 16, OK), (65535 * 16 + 1, OK), (65535 * 32, OK), (65535 * 32 + 1, OK),
                                         (65535 * 64, OK), (65535 * 64 + 1, UNSUPPORTED)])
def test_rows_of_one_4_bit_weight(n, k, rows, status):
    assert w4_status(rows, n, k) == status


@pytest.mark.parametrize("rows,matrices,n,k,status", [
    (65535 * 16, 16, 16, 1024, OK), (1 << 21, 16, 32, 4096, OK),   # the model's choice has 16 or 32 rows a block
    (200_000, 60_000, 64, 128, OK),                                # up to four rows a matrix
    (900_000, 60_000, 1024, 256, UNSUPPORTED), (600_000, 50_000, 1024, 256, OK),  # many blocks of up to 16 rows
    (70_000, 70_000, 16, 128, UNSUPPORTED)])                       # a block for each row
def test_rows_of_4_bit_experts(rows, matrices, n, k, status):
    assert w4_status(rows, n, k, matrices, offsets=True) == status
