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


# Sizes whose byte counts would pass 64 bits: no such operand exists, and the counts came out small or negative
@pytest.mark.parametrize("matrices,n,k,status", [
    (1 << 24, 1 << 24, 1 << 24, UNSUPPORTED), (1 << 24, 1 << 24, 1 << 20, UNSUPPORTED), (1 << 24, 16, 128, OK),
    (1, 1 << 24, 1 << 24, OK), (256, 1 << 24, 1 << 24, OK), (257, 1 << 24, 1 << 24, UNSUPPORTED)])
@pytest.mark.parametrize("group,zeros", [(32, 1), (128, 0)])
def test_bytes_of_4_bit_weights(matrices, n, k, status, group, zeros):
    b = ctypes.c_int64(-5)
    assert spt.lib().gemm_w4_packed_bytes(matrices, n, k, group, zeros, ctypes.byref(b)) == status
    if status == OK:
        assert b.value == matrices * -(-n // 16) * -(-k // 128) * (1024 + 16 * 128 // group * (2 + zeros))
    else:
        assert spt.lib().gemm_w4_pack(0x1000, 0x1000, None, matrices, n, k, group, 0x1000, None) == UNSUPPORTED
        assert w4_status(4, n, k, matrices, offsets=True) == UNSUPPORTED


@pytest.mark.parametrize("mode", [_lib.GEMM_GROUPED_FORWARD, _lib.GEMM_GROUPED_GRAD_A, _lib.GEMM_GROUPED_GRAD_B])
@pytest.mark.parametrize("change,status", [
    (dict(experts=2**31 - 1, n=2**19 + 1, stride=2**39, ld=2**19 + 1), UNSUPPORTED),
    (dict(experts=2**31 - 1, n=2**19 + 1, stride=2**62, ld=2**19 + 1), UNSUPPORTED), (dict(stride=2**63 - 1), UNSUPPORTED),
    (dict(experts=1, stride=2**63 - 1), UNSUPPORTED), (dict(stride=2**40), OK),
    (dict(n=2**19 + 1, ld=2**62, stride=2**40), UNSUPPORTED)])  # rows of the matrices too far apart for the products
def test_bytes_of_experts(mode, change, status):
    c = dict(experts=4, n=32, stride=32 * 48, ld=48)
    c.update(change)
    gb = mode == _lib.GEMM_GROUPED_GRAD_B
    wide = 2**19 + 1  # at least n and k
    p = _lib.GemmGrouped(mode=mode, rows=3, experts=c["experts"], n=c["n"], k=min(c["ld"], 48), in_dtype=BF16, out_dtype=BF16,
                         ldx=wide, ldy=wide if gb else c["ld"], ldo=c["ld"] if gb else wide, stride=c["stride"], tile=256)
    b = ctypes.c_int64(0)
    got = spt.lib().gemm_grouped_workspace_bytes(ctypes.byref(p), 0x1000, 0x1000, ctypes.byref(b))
    assert got == status and b.value >= 0


@pytest.mark.parametrize("experts,status", [(1 << 24, OK), ((1 << 24) + 1, UNSUPPORTED), (2**31 - 1, UNSUPPORTED)])
def test_number_of_experts(experts, status):
    # the search for a tile's expert counts experts, and the rows of nobody, in 32 bits
    p = _lib.GemmGrouped(mode=0, rows=3, experts=experts, n=1, k=1, in_dtype=BF16, out_dtype=BF16, ldx=1, ldy=1, ldo=1, stride=1)
    b = ctypes.c_int64(0)
    assert spt.lib().gemm_grouped_workspace_bytes(ctypes.byref(p), 0x1000, 0x1000, ctypes.byref(b)) == status
    assert w4_status(3, 16, 128, experts, offsets=True) == status
