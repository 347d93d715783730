"""Microscaled operators and the norm where offsets pass 32 bits: the far end of a large tensor gives what the same rows give
by themselves. Values are eighths, so that sums are exact whichever kernel has them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TALL, WIDE = 70_001, 65_536  # 2^32 bytes of 8-bit codes, and some


@pytest.fixture(scope="module", autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def operand(rows, k, bits, seed):
    """1, 1.125 .. 1.5 in 8 bits (65536 products of two: below 2^24 units of 2^-6), or any of the 4-bit codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    low, high = (0x38, 0x3D) if bits == 8 else (0, 256)
    codes = torch.randint(low, high, (rows, k * bits // 8), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")
    return spt.pack_mx(codes, scales, bits, k), codes, scales


@pytest.mark.parametrize("big", ["a", "b"])
@pytest.mark.parametrize("small", [8, 64, 300])
def test_products_of_large_operands(big, small):
    q, codes, scales = operand(TALL, WIDE, 8, 1)
    few, _, _ = operand(small, WIDE, 8, 2)
    end = slice(TALL - 70, TALL)
    tail = spt.pack_mx(codes[end], scales[end], 8)
    if big == "a":
        got, want = spt.mx_matmul(q, few, BF16)[end], spt.mx_matmul(tail, few, BF16)
    else:
        got, want = spt.mx_matmul(few, q, BF16)[:, end], spt.mx_matmul(few, tail, BF16)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [(8, 8), (8, 4), (4, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_results(bits, dtype):
    m, n = TALL, 40_000
    a, ca, sa = operand(m, 128, bits[0], 1)
    b, cb, sb = operand(n, 128, bits[1], 2)
    c = spt.mx_matmul(a, b, dtype)
    rows, cols = slice(m - 100, m), slice(n - 100, n)
    a2, b2 = spt.pack_mx(ca[rows], sa[rows], bits[0]), spt.pack_mx(cb[cols], sb[cols], bits[1])
    assert torch.equal(c[rows, cols], spt.mx_matmul(a2, b2, dtype))
    assert torch.equal(c[rows], spt.mx_matmul(a2, b, dtype))


@pytest.mark.parametrize("bits", [4, 8])
def test_large_quantised_tensors(bits):
    x = torch.randn((TALL, WIDE), dtype=BF16, device="cuda")
    end = slice(TALL - 130, TALL)
    q, tail = spt.quantize_mx(x, bits), spt.quantize_mx(x[end], bits)
    assert torch.equal(q.codes[end], tail.codes)
    want = spt.dequantize_mx(tail)
    assert torch.equal(spt.dequantize_mx(q, out=x)[end], want)


def test_norm_of_a_large_tensor():
    x = torch.randn((TALL, WIDE // 2), dtype=BF16, device="cuda")
    r = torch.randn((TALL, WIDE // 2), dtype=BF16, device="cuda")
    w = torch.rand(WIDE // 2, device="cuda")
    end = slice(TALL - 130, TALL)
    y, h = spt.rms_norm(x, w, residual=r)
    y2, h2 = spt.rms_norm(x[end], w, residual=r[end])
    assert torch.equal(y[end], y2) and torch.equal(h[end], h2)
    q, q2 = spt.rms_norm_mx(h, w), spt.rms_norm_mx(h2, w)
    assert torch.equal(q.codes[end], q2.codes)
    dx, _ = spt.rms_norm_grad(x, h, w, dh=r)
    assert torch.equal(dx[end], spt.rms_norm_grad(x[end], h2, w, dh=r[end])[0])
