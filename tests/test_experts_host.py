"""The experts' operators and 4-bit weights on a host without a GPU: the header's symbols are exported and
bound, and every refusal the C ABI and the torch face make before any device work."""
import ctypes
import os
import re

import pytest
import torch

import software_pipelined_tiled_amd as spt
from software_pipelined_tiled_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = _lib.GEMM_OK, _lib.GEMM_ERR_INVALID, _lib.GEMM_ERR_UNSUPPORTED
F16, BF16, F32 = spt.GEMM_F16, spt.GEMM_BF16, spt.GEMM_F32
A = 0x1000  # a non-null, 16-byte aligned address that no refused call reads


def test_library_exports_every_header_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "experts.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"gemm_status_t\s+(\w+)\s*\(", text)))
    assert names == sorted(spt.EXPERT_EXPORTS)
    for n in names:
        assert hasattr(spt.lib(), n), n


def test_enum_values_match_the_header():
    text = open(os.path.join(ROOT, "include", "experts.h")).read()
    for name in ("FORWARD", "GRAD_A", "GRAD_B"):
        value = int(re.search(rf"GEMM_GROUPED_{name}\s*=\s*(\d+)", text).group(1))
        assert value == getattr(_lib, f"GEMM_GROUPED_{name}")


@pytest.mark.parametrize("slots,experts,want", [
    (0, 1, 0), (4096, 8, 0), (4097, 8, 5 * 9 * 4), (1 << 20, 1024, 256 * 1025 * 4), (2**31 - 1, 4, None)])
def test_sort_workspace(slots, experts, want):
    got = spt._lib.experts_sort_workspace_bytes(slots, experts)
    if want is not None:
        assert got == want
    assert got <= 257 * (experts + 1) * 4  # never more than 256 workgroups and one of rounding


@pytest.mark.parametrize("slots,experts,status", [
    (-1, 4, INVALID), (5, 0, UNSUPPORTED), (5, -3, UNSUPPORTED), (5, 1025, UNSUPPORTED), (2**31, 4, UNSUPPORTED)])
def test_sort_workspace_refusals(slots, experts, status):
    n = ctypes.c_int64()
    assert spt.lib().experts_sort_workspace_bytes(slots, experts, ctypes.byref(n)) == status
    assert spt.lib().experts_sort_workspace_bytes(4, 4, None) == INVALID


@pytest.mark.parametrize("args", [
    (A, 16, 4, 4, A, A, A, None, 0), (None, 32, 4, 4, A, A, A, None, 0), (A, 32, 4, 4, None, A, A, None, 0),
    (A, 32, 4, 4, A, None, A, None, 0), (A, 32, 4, 4, A, A, None, None, 0),
    (A, 64, 9000, 4, A, A, A, None, 0), (A, 64, 9000, 4, A, A, A, A, 59)])
def test_sort_refusals(args):
    assert spt.lib().experts_sort(*args, None) == INVALID


@pytest.mark.parametrize("args,status", [
    ((A, 3, 4, 2, 8, 8, A, A, A, 8), INVALID), ((A, F16, -4, 2, 8, 8, A, A, A, 8), INVALID),
    ((A, F16, 4, 2, 8, 7, A, A, A, 8), INVALID), ((A, F16, 4, 2, 8, 8, A, A, A, 7), INVALID),
    ((None, F16, 4, 2, 8, 8, A, A, A, 8), INVALID), ((A, F16, 4, 2, 8, 8, None, A, A, 8), INVALID),
    ((A, F16, 4, 2, 8, 8, A, None, A, 8), INVALID), ((A, F16, 4, 2, 8, 8, A, A, None, 8), INVALID),
    ((A, F16, 2**30, 2, 8, 8, A, A, A, 8), UNSUPPORTED), ((A, F16, 2**30, 1, 2048, 2048, A, A, A, 2048), UNSUPPORTED),
    ((A, F16, 0, 2, 8, 8, None, None, None, 8), OK), ((A, F32, 4, 2, 0, 8, None, None, None, 8), OK)])
def test_gather_refusals(args, status):
    assert spt.lib().experts_gather(*args, 1, None) == status


@pytest.mark.parametrize("args,status", [
    ((A, 5, 4, 2, 8, 8, A, A, None, 0, A, 8), INVALID), ((A, BF16, 4, 2, 8, 8, A, A, A, 7, A, 8), INVALID),
    ((None, BF16, 4, 2, 8, 8, A, A, None, 0, A, 8), INVALID), ((A, BF16, 4, 2, 8, 8, A, None, None, 0, A, 8), INVALID),
    ((A, BF16, 4, 2, 8, 4, A, A, None, 0, A, 8), INVALID), ((A, BF16, 0, 2, 8, 8, None, None, None, 0, None, 8), OK)])
def test_combine_refusals(args, status):
    assert spt.lib().experts_combine(*args, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=9), INVALID), (dict(lddo=3), INVALID), (dict(ldy=3), INVALID), (dict(lddy=3), INVALID),
    (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(dy=None), INVALID), (dict(rows=None), INVALID),
    (dict(dw=None), INVALID), (dict(wdtype=4), INVALID), (dict(tokens=2**23, top_k=1), UNSUPPORTED), (dict(tokens=0), OK)])
def test_combine_grad_refusals(change, status):
    a = dict(dout=A, lddo=8, y=A, dtype=F16, tokens=4, top_k=2, width=8, ldy=8, rows=A, kept=A, w=A, wdtype=F32, dy=A,
             lddy=8, dw=A, rest=1)
    a.update(change)
    assert spt.lib().experts_combine_grad(*a.values(), None) == status


def grouped(**change):
    p = dict(mode=0, rows=64, experts=4, n=32, k=48, in_dtype=BF16, out_dtype=BF16, ldx=48, ldy=48, ldo=32, stride=32 * 48,
             zero_rest=0)
    p.update(change)
    return _lib.GemmGrouped(**p)


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(mode=3), INVALID), (dict(mode=-1), INVALID), (dict(rows=-1), INVALID), (dict(n=-1), INVALID),
    (dict(experts=-1), INVALID), (dict(in_dtype=7), INVALID), (dict(out_dtype=7), INVALID), (dict(in_dtype=F32), UNSUPPORTED),
    (dict(ldx=47), INVALID), (dict(ldy=47), INVALID), (dict(ldo=31), INVALID), (dict(stride=31 * 48 + 47), INVALID),
    (dict(stride=0, experts=1), OK), (dict(rows=2**31), UNSUPPORTED), (dict(ldx=2**20), UNSUPPORTED),
    (dict(ldy=2**20, stride=2**26), UNSUPPORTED), (dict(ldo=2**20), UNSUPPORTED),
    (dict(mode=1, ldx=31, ldo=48), INVALID), (dict(mode=1, ldx=32, ldo=47), INVALID), (dict(mode=1, ldx=32, ldo=48), OK),
    (dict(mode=2, ldx=32, ldo=47), INVALID), (dict(mode=2, ldx=32, ldo=48), OK),
    (dict(tile=64), INVALID), (dict(tile=32), OK), (dict(tile=32, mode=2, ldx=32, ldo=48), UNSUPPORTED), (dict(tile=256), OK)])
def test_grouped_shapes(change, status):
    n = ctypes.c_int64()
    assert spt.lib().gemm_grouped_workspace_bytes(ctypes.byref(grouped(**change)), A, A, ctypes.byref(n)) == status


def test_grouped_workspace_is_for_operands_off_sixteen_bytes():
    # only the 256-row tiles copy an operand; the others load any alignment
    def ws(x=A, y=A, **change):
        return _lib.gemm_grouped_workspace_bytes(grouped(**{"tile": 256, **change}), x, y)
    assert ws() == 0
    assert ws(x=A + 2) == 64 * 48 * 2                      # A copied
    assert ws(x=A + 2, tile=128) == ws(x=A + 2, tile=32) == 0
    assert ws(y=A + 8) == 4 * 32 * 48 * 2                  # B copied
    assert ws(ldx=50) == 64 * 48 * 2
    assert ws(k=45, ldx=45, ldy=45, stride=32 * 45) == (64 + 4 * 32) * 48 * 2  # rows of 45 padded to 48
    assert ws(mode=2, ldx=33, n=33, ldo=48, stride=33 * 48) == 64 * 40 * 2
    # the library's choice: a large B is not copied for a few rows
    assert ws(tile=0, rows=5000, experts=64, n=1409, k=2044, ldx=2044, ldy=2044, ldo=1409, stride=1409 * 2044) == 0


def test_grouped_run_refusals():
    L, p = spt.lib(), grouped(tile=256)
    assert L.gemm_grouped_run(None, A, A, A, A, None, 0, None) == INVALID
    assert L.gemm_grouped_run(ctypes.byref(p), None, A, A, A, None, 0, None) == INVALID
    assert L.gemm_grouped_run(ctypes.byref(p), A, None, A, A, None, 0, None) == INVALID
    assert L.gemm_grouped_run(ctypes.byref(p), A, A, None, A, None, 0, None) == INVALID
    assert L.gemm_grouped_run(ctypes.byref(p), A, A, A, None, None, 0, None) == INVALID
    assert L.gemm_grouped_run(ctypes.byref(p), A + 2, A, A, A, None, 0, None) == INVALID         # workspace missing
    assert L.gemm_grouped_run(ctypes.byref(p), A + 2, A, A, A, A, 64 * 48 * 2 - 1, None) == INVALID  # too small
    assert L.gemm_grouped_run(ctypes.byref(grouped(rows=0)), None, A, A, A, None, 0, None) == OK  # nothing to do
    assert L.gemm_grouped_run(ctypes.byref(grouped(n=0, stride=0, ldo=0)), A, None, None, A, None, 0, None) == OK


@pytest.mark.parametrize("args,status", [
    ((1, 16, 128, 128, 0), OK), ((1, 16, 128, 16, 0), UNSUPPORTED), ((1, 16, 128, 48, 0), UNSUPPORTED),
    ((-1, 16, 128, 32, 0), INVALID), ((1, -1, 128, 32, 0), INVALID), ((1, 16, -1, 32, 0), INVALID),
    ((1, 2**24 + 1, 128, 32, 0), UNSUPPORTED), ((1, 16, 2**24 + 1, 32, 0), UNSUPPORTED)])
def test_w4_packed_bytes_refusals(args, status):
    n = ctypes.c_int64()
    assert spt.lib().gemm_w4_packed_bytes(*args, ctypes.byref(n)) == status


def test_w4_packed_bytes():
    f = _lib.gemm_w4_packed_bytes
    assert f(1, 16, 128, 128, False) == 1024 + 32
    assert f(1, 16, 128, 32, True) == 1024 + 128 + 64
    assert f(3, 17, 129, 64, False) == 3 * 2 * 2 * (1024 + 64)  # columns to 16, k to 128
    assert f(0, 16, 128, 64, False) == f(2, 0, 128, 64, True) == f(2, 16, 0, 64, True) == 0


def test_w4_pack_refusals():
    L = spt.lib()
    assert L.gemm_w4_pack(None, A, None, 1, 16, 128, 64, A, None) == INVALID
    assert L.gemm_w4_pack(A, None, None, 1, 16, 128, 64, A, None) == INVALID
    assert L.gemm_w4_pack(A, A, None, 1, 16, 128, 64, None, None) == INVALID
    assert L.gemm_w4_pack(A, A, None, 1, 16, 128, 64, A + 8, None) == INVALID
    assert L.gemm_w4_pack(A, A, None, 1, 16, 128, 63, A, None) == UNSUPPORTED
    assert L.gemm_w4_pack(None, None, None, 0, 16, 128, 64, None, None) == OK


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(dtype=F32), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(group=16), UNSUPPORTED), (dict(ldx=127), INVALID), (dict(ldo=15), INVALID), (dict(matrices=2), INVALID),
    (dict(ldx=2**23), UNSUPPORTED), (dict(n=2**24 + 1, ldo=2**25), UNSUPPORTED), (dict(rows=2**23), UNSUPPORTED),
    (dict(rows=0), OK), (dict(n=0), OK)])
def test_w4_run_refusals(change, status):
    p = dict(rows=4, matrices=1, n=16, k=128, group=64, has_zeros=0, dtype=F16, out_dtype=F16, ldx=128, ldo=16, zero_rest=0)
    p.update(change)
    assert spt.lib().gemm_w4_run(ctypes.byref(_lib.GemmW4(**p)), A, A, None, A, None, 0, None) == status


def test_w4_run_null_operands():
    p = _lib.GemmW4(rows=4, matrices=1, n=16, k=128, group=64, has_zeros=0, dtype=F16, out_dtype=F16, ldx=128, ldo=16)
    run = spt.lib().gemm_w4_run
    assert run(None, A, A, None, A, None, 0, None) == INVALID
    assert run(ctypes.byref(p), None, A, None, A, None, 0, None) == INVALID
    assert run(ctypes.byref(p), A, None, None, A, None, 0, None) == INVALID
    assert run(ctypes.byref(p), A, A + 4, None, A, None, 0, None) == INVALID
    assert run(ctypes.byref(p), A, A, None, None, None, 0, None) == INVALID


def test_torch_face_wants_device_tensors():
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    order = spt.TokenOrder(torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                           torch.zeros((4, 2), dtype=torch.int32), 2)
    off = torch.zeros(3, dtype=torch.int32)
    b = torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    for call in (lambda: spt.sort_tokens(torch.zeros((4, 2), dtype=torch.int64), 2),
                 lambda: spt.gather_rows(t, order), lambda: spt.combine_rows(t.repeat(2, 1), order),
                 lambda: spt.gather_rows_grad(t.repeat(2, 1), order),
                 lambda: spt.combine_rows_grad(t, t.repeat(2, 1), order),
                 lambda: spt.grouped_matmul(t, b, off), lambda: spt.grouped_matmul_grad_a(t, b, off),
                 lambda: spt.grouped_matmul_grad_b(t, t, off),
                 lambda: spt.pack_w4(torch.zeros((8, 32), dtype=torch.uint8), t[:, :1].repeat(2, 1), group_size=32),
                 lambda: spt.routed_matmul(t, b, torch.zeros((4, 2), dtype=torch.int64))):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_torch_face_wants_supported_types():
    t = torch.zeros((4, 8))
    with pytest.raises(TypeError):
        spt.sort_tokens(torch.zeros((4, 2), dtype=torch.int16), 2)
    with pytest.raises(TypeError):
        spt.grouped_matmul(t, torch.zeros((2, 8, 8)), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        spt.grouped_matmul_grad_b(t, t, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        spt.pack_w4(torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 1)), group_size=32)
    with pytest.raises(ValueError):
        spt.pack_w4(torch.zeros((8, 32), dtype=torch.int8), torch.zeros((8, 1), dtype=torch.float16), group_size=32)


def test_too_many_output_tiles():
    # 2^22 row blocks of 256 by 8 column tiles
    p = grouped(rows=2**30, experts=1, n=2048, k=8, ldx=8, ldy=8, ldo=2048, stride=2048 * 8, tile=256)
    assert spt.lib().gemm_grouped_run(ctypes.byref(p), A, A, A, A, None, 0, None) == UNSUPPORTED


def test_token_order_checks_its_parts():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    assert spt.TokenOrder(i32(4), i32(6), i32(3, 2), 3).sorted_rows == 6
    for bad in ((i32(3), i32(6), i32(3, 2)), (i32(4), i32(5), i32(3, 2)), (i32(4), i32(6), i32(6)),
                (i32(4), i32(6), i32(2, 3).t()), (i32(4).long(), i32(6), i32(3, 2)), (i32(4), i32(6), i32(3, 2).long())):
        with pytest.raises(ValueError):
            spt.TokenOrder(*bad, 3)


def test_w4_weight_checks_its_bytes():
    make = lambda size, stacked=False, m=1: spt.W4Weight(torch.zeros(size, dtype=torch.uint8), m, stacked, 17, 129, 64, False,
                                                         torch.float16)
    assert make(2 * 2 * (1024 + 64)).n == 17
    for bad in (lambda: make(2 * 2 * (1024 + 64) - 1), lambda: make(0), lambda: make(2 * 4 * (1024 + 64), False, 2)):
        with pytest.raises(ValueError, match="packed"):
            bad()


def test_routed_matmul_shapes():
    x, b = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    ids = torch.zeros((4, 2), dtype=torch.int64)
    for bad in ((x[0], b, ids), (x, b[0], ids), (x, b, ids[0, 0]), (x, b, ids[:3])):
        with pytest.raises(ValueError):
            spt.routed_matmul(*bad)


def test_w4_workspace_and_refusals_of_it():
    def ws(has_offsets=False, **change):
        p = dict(rows=4, matrices=1, n=16, k=128, group=64, has_zeros=0, dtype=F16, out_dtype=F16, ldx=128, ldo=16, zero_rest=0)
        p.update(change)
        return _lib.gemm_w4_workspace_bytes(_lib.GemmW4(**p), has_offsets)
    assert ws() == 0  # one block of K
    assert ws(k=4096, ldx=4096) == 4 * 4 * 16 * 4  # 32 blocks over eight waves: four parts
    assert ws(n=8192, ldo=8192, k=8192, ldx=8192) == 0  # columns enough
    with pytest.raises(_lib.GemmError):
        ws(matrices=2)
    p = _lib.GemmW4(rows=4, matrices=1, n=16, k=4096, group=64, has_zeros=0, dtype=F16, out_dtype=F16, ldx=4096, ldo=16)
    for workspace, size in ((None, 0), (A, 1023), (A + 2, 2048)):
        assert spt.lib().gemm_w4_run(ctypes.byref(p), A, A, None, A, workspace, size, None) == INVALID


def test_grouped_workspace_of_cut_sums():
    def ws(**change):
        return _lib.gemm_grouped_workspace_bytes(grouped(**{"rows": 2, "k": 4096, "ldx": 4096, "ldy": 4096, "stride": 32 * 4096,
                                                            **change}), A, A)
    assert ws() == 8 * 2 * 32 * 4                       # two tiles, 64 K-tiles: parts of eight
    assert ws(tile=128) == 0 and ws(k=1024) == 0
    assert ws(n=8192, ldo=8192, stride=8192 * 4096) == 2 * 2 * 8192 * 4  # 256 tiles: two parts
    assert ws(rows=4, n=8192, ldo=8192, stride=8192 * 4096) == 0         # 512: tiles enough
    p = grouped(rows=2, k=4096, ldx=4096, ldy=4096, stride=32 * 4096)
    for workspace, size in ((None, 0), (A, 8 * 2 * 32 * 4 - 1), (A + 4, 1 << 20)):
        assert spt.lib().gemm_grouped_run(ctypes.byref(p), A, A, A, A, workspace, size, None) == INVALID
