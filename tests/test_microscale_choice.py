"""Which kernel a microscaled product takes, on a host without a GPU: what is reported, and that the GPU tests' shapes take all of them."""
import ast
import ctypes
import math
import os
import random

import pytest

import software_pipelined_tiled_amd as spt
from microscale_cases import FORMATS, REAL
from software_pipelined_tiled_amd import _lib

TYPES = (spt.GEMM_F16, spt.GEMM_BF16, spt.GEMM_F32)


def choice(m, n, k, fa, fb, out):
    return _lib.gemm_mx_describe(_lib.GemmMx(m, n, k, fa, fb, out, max(n, 1)))


def kinds(shapes):
    """(formats, result type, kernel, rows of its tile, whether its sum is in parts) of all shapes in all formats and types."""
    found = set()
    for m, n, k in shapes:
        for fa, fb in FORMATS:
            for out in TYPES:
                c = choice(m, n, k, fa, fb, out)
                found.add((fa, fb, out, c["kernel"], c["bm"], c["splits"] > 1))
    return found


def some_shapes(count, k_from, seed):
    rng = random.Random(seed)
    draw = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    return [(draw(1, 20000), draw(1, 30000), draw(k_from, 40000)) for _ in range(count)]


def test_shapes_of_the_tests_take_every_kernel():
    path = os.path.join(os.path.dirname(__file__), "test_microscale_gpu.py")
    lists = {}
    for node in ast.walk(ast.parse(open(path).read())):
        if isinstance(node, ast.FunctionDef) and node.name == "test_matmul_every_kernel":
            for d in node.decorator_list:
                if ast.literal_eval(d.args[0]) == "m,n,k":
                    lists["exact"] = ast.literal_eval(d.args[1])
    assert len(lists["exact"]) > 10
    assert kinds(some_shapes(20000, 1, 1)) <= kinds(lists["exact"])
    assert kinds(some_shapes(20000, 300, 2)) <= kinds(REAL)


def test_every_kernel_is_among_them():
    """Few rows by 16 and 32, tiles of 32, 64 and 128 rows, and, but for fp32 results of 8-bit operands, two groups of waves."""
    of = {}
    for fa, fb, out, kernel, bm, split in kinds(REAL):
        of.setdefault((fa, fb, out), set()).add((kernel, bm, split))
    for (fa, fb, out), found in of.items():
        tiles = {(1, bm, split) for bm in (32, 64, 128) for split in (False, True)}
        two = set() if out == spt.GEMM_F32 and fa == 8 else {(2, 256, False), (2, 256, True)}
        # of two formats few rows go to the 32-row kernel by itself only in between
        assert tiles | two | {(0, 16, False)} <= found <= tiles | two | {(0, 16, False), (0, 32, False)}, (fa, fb, out)


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("out", TYPES)
def test_description(fa, fb, out):
    for m, n, k in some_shapes(500, 1, 3) + [(1, 1, 1), (5, 7, 0), (0, 5, 100), (5, 0, 100)]:
        p = _lib.GemmMx(m, n, k, fa, fb, out, max(n, 1))
        c = choice(m, n, k, fa, fb, out)
        assert c["through_bf16"] == (out == spt.GEMM_F32 and fa == 8)
        assert c["bm"] in ((16, 32), (32, 64, 128), (256,))[c["kernel"]] and c["bn"] == (16, 128, 256)[c["kernel"]]
        assert c["k_per_part"] % 128 == 0 and 1 <= c["splits"] <= 16
        if min(m, n, k):
            assert (c["splits"] - 1) * c["k_per_part"] < k <= c["splits"] * c["k_per_part"]
            assert _lib.gemm_mx_workspace_bytes(p) == (c["splits"] * m * n * 4 if c["splits"] > 1 else 0)
            if c["kernel"] == 2:  # its pipeline has two K-tiles or more in every part
                kt = 256 if fa == 4 else 128
                assert -(-(k - (c["splits"] - 1) * c["k_per_part"]) // kt) >= 2


def test_refusals():
    size = ctypes.byref(_lib.GemmMxConfig())
    for change, status in ((dict(m=-1), _lib.GEMM_ERR_INVALID), (dict(a_bits=4), _lib.GEMM_ERR_UNSUPPORTED), (dict(ldc=3), _lib.GEMM_ERR_INVALID)):
        p = _lib.GemmMx(*({**dict(m=4, n=5, k=6, a_bits=8, b_bits=8, out_dtype=0, ldc=5), **change}[f] for f, _ in _lib.GemmMx._fields_))
        assert spt.lib().gemm_mx_describe(ctypes.byref(p), size) == status
    p = _lib.GemmMx(4, 5, 6, 8, 8, 0, 5)
    assert spt.lib().gemm_mx_describe(ctypes.byref(p), None) == _lib.GEMM_ERR_INVALID
    assert spt.lib().gemm_mx_describe(None, size) == _lib.GEMM_ERR_INVALID
