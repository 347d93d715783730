"""The norm and the microscaled products as a model uses them together: a decoding loop over layers with the residual stream in one
tensor, eager and as a replayed graph, and a training step through the norm beside torch's own operators."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def rand(*shape, dtype=BF16, seed=0, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(dtype)


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
@pytest.mark.parametrize("bits,wbits", [(8, 8), (8, 4), (4, 4)])
def test_decoding_loop(rows, bits, wbits):
    """Layers of norm with residual, up product, quantisation, down product: the calls in place and captured give the bits of the calls
    that make new tensors."""
    d, f, layers = 512, 1408, 3
    up = [spt.quantize_mx(rand(f, d, seed=10 + i, scale=d**-0.5), wbits) for i in range(layers)]
    down = [spt.quantize_mx(rand(d, f, seed=20 + i, scale=f**-0.5), wbits) for i in range(layers)]
    gain = [1 + rand(d, dtype=F32, seed=30 + i, scale=0.1) for i in range(layers)]

    def plain(x):
        stream, out = x, torch.zeros_like(x)
        for i in range(layers):
            _, stream = spt.rms_norm(out, gain[i], residual=stream)
            q = spt.rms_norm_mx(stream, gain[i], bits=bits)
            a = torch.relu(spt.mx_matmul(q, up[i]))
            out = spt.mx_matmul(spt.quantize_mx(a, bits), down[i])
        return out, stream

    def in_place(x, stream, out):
        stream.copy_(x)
        out.zero_()
        for i in range(layers):
            q, _ = spt.rms_norm_mx(out, gain[i], residual=stream, bits=bits, residual_out=stream)
            a = torch.relu_(spt.mx_matmul(q, up[i]))
            spt.mx_linear(a, down[i], bits, out=out)

    x = rand(rows, d, seed=1)
    stream, out = torch.empty_like(x), torch.empty_like(x)
    in_place(x, stream, out)
    want = plain(x)
    assert torch.equal(out, want[0]) and torch.equal(stream, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        in_place(x, stream, out)
    for turn in range(4):
        x.copy_(rand(rows, d, seed=100 + turn))
        g.replay()
        want = plain(x)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(stream, want[1]), turn


def test_training_step():
    """Two layers of norm with residual and product, in fp32 against the same in 64 bits. Sums have at most 160 terms, each off by less
    than 160 * 2^-24 < 2^-16 of its terms' magnitudes; some ten of them follow each other, and in the 2-norm of random values the
    terms' magnitudes exceed the sums by less than 2^4: 2^-8 of each gradient's norm bounds them all."""
    rows, d, f = 37, 96, 160
    shapes = [(rows, d), (d,), (d, f), (d,), (f, d), (d,)]
    leaves = [rand(*s, dtype=F32, seed=i, scale=1.0 if len(s) == 2 and s[0] == rows else 0.2) + (1.0 if len(s) == 1 else 0.0)
              for i, s in enumerate(shapes)]
    leaves = [t.requires_grad_() for t in leaves]

    def step(x, g1, w1, g2, w2, g3, norm):
        stream, out = x, torch.zeros_like(x)
        y, stream = norm(out, g1, stream)
        out = torch.tanh(y @ w1) @ w2
        y, stream = norm(out, g2, stream)
        out = torch.tanh(y @ w1) @ w2
        y, stream = norm(out, g3, stream)
        return y.square().sum() * 0.5 + (stream * y).sum()

    def reference(x, g, r):
        h = x + r
        return h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * g, h

    got = torch.autograd.grad(step(*leaves, lambda x, g, r: spt.rms_norm(x, g, 1e-6, residual=r)), leaves)
    wide = [t.detach().to(F64).requires_grad_() for t in leaves]
    want = torch.autograd.grad(step(*wide, reference), wide)
    for a, b in zip(got, want):
        assert ((a.to(F64) - b).norm() <= 2.0**-8 * b.norm()).item()
