"""A captured backward pass that would reach a gradient accumulator of the
default stream (an eager graph of the same leaf lives) is refused by every
differentiable call, whatever lies between the call and the leaf; what reaches
none, or only captures the forward pass, runs."""
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

M, K, F = 40, 64, 96


def bf16(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def calls(b):
    x, w, both = bf16(M, K), bf16(F, K, seed=1), bf16(2 * F, K, seed=2)
    # the leaf, and what is computed from it; none is refused in the forward pass
    return {
        "fake_quant nvfp4": (w, lambda t: b.fake_quant(t)),
        "qat_linear nvfp4, weight": (w, lambda t: b.qat_linear(x, t)),
        "qat_linear nvfp4, input": (x, lambda t: b.qat_linear(t, w)),
        "qat_linear nvfp4, quantized input": (x, lambda t: b.qat_linear(t, w, act_quant=True)),
        "qat_linear mxfp4, input": (x, lambda t: b.qat_linear(t, w, fmt="mxfp4")),
        "qat_linear mxfp4, view": (both, lambda t: b.qat_linear(x, t[:F], fmt="mxfp4")),
        "gated_linear, views": (both, lambda t: b.gated_linear(x, t[:F], t[F:])),
        "qat_gated_linear, views": (both, lambda t: b.qat_gated_linear(x, t[:F], t[F:], fmt="mxfp4")),
    }


NAMES = ["fake_quant nvfp4", "qat_linear nvfp4, weight", "qat_linear nvfp4, input", "qat_linear nvfp4, quantized input",
         "qat_linear mxfp4, input", "qat_linear mxfp4, view", "gated_linear, views", "qat_gated_linear, views"]


@pytest.mark.parametrize("name", NAMES)
def test_captured_backward_beside_an_eager_graph_is_refused(name):
    b = need_gpu()
    leaf, run = calls(b)[name]
    leaf = leaf.clone().requires_grad_(True)
    eager = run(leaf)
    ref, g = eager.detach().clone(), torch.ones_like(eager)
    other = leaf.detach().clone().requires_grad_(True)
    torch.autograd.grad(run(other), other, g)      # (the products' library wants one pass before a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(leaf)
        with pytest.raises(RuntimeError, match="eager graph"):
            torch.autograd.grad(y, leaf, g)
        with pytest.raises(RuntimeError, match="eager graph"):
            run(leaf).backward(g)
    graph.replay()                                                     # the forward pass was captured
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and leaf.grad is None
    (want,) = torch.autograd.grad(eager, leaf, g)                      # the eager graph is intact
    del eager, y
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(leaf)
        (got,) = torch.autograd.grad(y, leaf, g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and torch.equal(got, want) and b.stream_status() == 0


@pytest.mark.parametrize("name", ["fake_quant nvfp4", "gated_linear, views"])
def test_gradient_that_stops_short_of_the_leaf_is_captured(name):
    b = need_gpu()
    leaf, run = calls(b)[name]
    leaf = leaf.clone().requires_grad_(True)
    eager = run(leaf * 1)
    g = torch.ones_like(eager)
    near = (leaf * 1).detach().requires_grad_(True)
    (want,) = torch.autograd.grad(run(near), near, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = leaf * 1
        (got,) = torch.autograd.grad(run(t), t, g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and eager.requires_grad and b.stream_status() == 0
