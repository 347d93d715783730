"""The norm in an autograd graph: what is saved and overwritten is seen, derivatives that the operators do not have are refused,
and captures beside living graphs; and calls on several streams and graphs."""
import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import software_pipelined_tiled_amd as spt  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# --------------------------------------------------------------------------------- what is saved

def test_the_saved_stream_changed_before_backward_is_seen():
    x, r, w = (rand(6, 96, seed=i).requires_grad_() for i in range(3))
    w = w[0].detach().clone().requires_grad_()
    y, h = spt.rms_norm(x, w, residual=r)
    with torch.no_grad():
        h.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y, h = spt.rms_norm(x, w, residual=r)
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", ["rms_norm", "residual_out", "rms_norm_mx", "dequantize_mx", "mx_matmul", "mx_linear"])
@pytest.mark.parametrize("view", [False, True])
def test_writing_a_saved_out_is_seen(name, view):
    x, r = rand(32, 128, seed=1), rand(32, 128, seed=2)
    q, wide = spt.quantize_mx(x), spt.quantize_mx(rand(128, 128, seed=3))
    calls = {"rms_norm": lambda o: spt.rms_norm(x, out=o), "residual_out": lambda o: spt.rms_norm(x, residual=r, residual_out=o),
             "rms_norm_mx": lambda o: spt.rms_norm_mx(x, residual=r, residual_out=o), "dequantize_mx": lambda o: spt.dequantize_mx(q, out=o),
             "mx_matmul": lambda o: spt.mx_matmul(q, wide, out=o), "mx_linear": lambda o: spt.mx_linear(x, wide, out=o)}
    buf = rand(32, 128, seed=4)
    leaf = rand(32, 128, seed=5).requires_grad_()
    loss = (leaf * buf).sum()
    with torch.no_grad():
        calls[name](buf[:, :] if view else buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_out_made_in_inference_mode():
    with torch.inference_mode():
        x = rand(4, 64)
        want = spt.rms_norm(x)
        assert torch.equal(spt.rms_norm(x, out=torch.empty_like(x)), want)
        q = spt.quantize_mx(x)
        assert torch.equal(spt.mx_matmul(q, q, out=torch.empty((4, 4), dtype=BF16, device="cuda")), spt.mx_matmul(q, q))


# ---------------------------------------------------------------------------- derivatives not there

@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_a_gradient_of_a_gradient_raises(which):
    args = [rand(8, 64, seed=1), rand(8, 64, seed=2), rand(1, 64, seed=3)[0].clone(), 1e-5, rand(8, 64, seed=4)]
    which = which if which < 3 else 4
    want = spt.rms_norm_grad(*args)
    leaf = args[which] = args[which].clone().requires_grad_()
    got = spt.rms_norm_grad(*args)
    for g, e in zip(got, want):
        assert torch.equal(g, e)
        with pytest.raises(RuntimeError, match="differentiable once"):
            (leaf.float().sum() + g.float().square().sum()).backward(retain_graph=True)
    with torch.no_grad():
        assert not any(g.requires_grad for g in spt.rms_norm_grad(*args))


def test_a_second_derivative_through_autograd_raises():
    x = rand(8, 64, seed=1).requires_grad_()
    g, = torch.autograd.grad(spt.rms_norm(x).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|differentiable once|twice"):
        g.float().sum().backward()


def test_tensors_that_require_grad():
    x, w = rand(8, 64).requires_grad_(), spt.quantize_mx(rand(16, 64))
    calls = [lambda: spt.quantize_mx(x), lambda: spt.rms_norm_mx(x), lambda: spt.rms_norm_mx(x.detach(), residual=x),
             lambda: spt.rms_norm_mx(x.detach(), x[0]), lambda: spt.mx_linear(x, w),
             lambda: spt.mx_matmul(w, w, out=rand(16, 16).requires_grad_()), lambda: spt.dequantize_mx(w, out=rand(16, 64).requires_grad_())]
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad():
            call()


def test_tensors_with_a_tangent():
    x, w = rand(8, 64), rand(1, 64)[0].clone()
    q = spt.quantize_mx(rand(8, 64))
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        bad = [lambda: spt.rms_norm(dual(x)), lambda: spt.rms_norm(x, dual(w)), lambda: spt.rms_norm(x, residual=dual(x)),
               lambda: spt.rms_norm(x, out=dual(x.clone())), lambda: spt.rms_norm_grad(x, dual(x)), lambda: spt.rms_norm_grad(x, x, dual(w)),
               lambda: spt.rms_norm_mx(x, dual(w)), lambda: spt.quantize_mx(dual(x)), lambda: spt.mx_linear(dual(x), q),
               lambda: spt.mx_matmul(q, q, out=dual(rand(8, 8))), lambda: spt.dequantize_mx(q, out=dual(x.clone()))]
        for call in bad:
            for mode in (torch.no_grad, torch.enable_grad):
                with mode(), pytest.raises(ValueError, match="forward-mode"):
                    call()
        leaf = x.clone().requires_grad_()
        y = spt.rms_norm(leaf)
        with pytest.raises(ValueError, match="forward-mode"):  # a gradient that arrives with a tangent
            torch.autograd.grad(y, leaf, dual(torch.ones_like(y)))


# -------------------------------------------------------------------------- streams and captures

@pytest.mark.parametrize("grad_mode", [False, True])
def test_gradients_of_leaves_captured_while_eager_ones_live(grad_mode):
    x, r, w = rand(300, 500, seed=1), rand(300, 500, seed=2).requires_grad_(), rand(1, 500, dtype=F32, seed=3)[0].clone().requires_grad_()
    dy = rand(300, 500, seed=4)
    with torch.no_grad():
        h = spt.rms_norm(x, w, residual=r)[1]
    alive = spt.rms_norm(x, w, residual=r)  # an eager graph of the same leaves

    def step():
        return spt.rms_norm_grad(dy, h, w, dh=dy)
    with torch.set_grad_enabled(grad_mode):
        eager = step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
    for rep in range(3):
        dy.mul_(1.5)
        g.replay()
        with torch.no_grad():
            want = step()
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            assert torch.equal(a, e), rep
    assert eager[0].requires_grad == grad_mode and got[1].requires_grad == grad_mode
    alive[0].sum().backward()
    assert w.grad is not None and r.grad is not None


def test_streams_and_two_graphs():
    """Calls on two streams at once, and two graphs replayed at once: each has workspaces of its own."""
    data = [(rand(2000, 1000, seed=i), rand(2000, 1000, seed=i + 9)) for i in range(2)]
    w = rand(1, 1000, dtype=F32, seed=3)[0].clone()
    want = [spt.rms_norm_grad(dy, h, w) for dy, h in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for turn in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(spt.rms_norm_grad(*data[i], w))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for dy, h in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(spt.rms_norm_grad(dy, h, w))
        graphs.append(g)
    for turn in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            got[i].append(tuple(t.clone() for t in outs[i]))
        torch.cuda.synchronize()
    for i in range(2):
        for dx, dw in got[i]:
            assert torch.equal(dx, want[i][0]) and torch.equal(dw, want[i][1])
