"""The rotation under autograd: the gradient of an input that asks for one."""

import pytest
import torch

from test_gpu_rope import BF, F32, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def positions(n):
    return torch.arange(n, dtype=torch.int32, device="cuda") * 37


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("grad", [False, True])
def test_an_input_gets_its_gradient(layout, dtype, grad):
    """The transposed rotation of the output's gradient, bit for bit, strided
    and broadcast ones too; of the transposed one the rotation."""
    import moe_expert_ffn_dg_gb300 as pkg
    rope = pkg.Rope(64, rot_dim=48, layout=layout, amplitude=1.3)
    pos = positions(5)
    x = torch.randn(5, 3, 64, device="cuda").to(dtype).requires_grad_()
    g = torch.randn(3, 5, 64, device="cuda").to(dtype).transpose(0, 1)
    y = rope.apply(x, pos, grad=grad)
    assert y.requires_grad and torch.equal(y.detach(), rope.apply(x.detach(), pos, grad=grad))
    got, = torch.autograd.grad(y, x, g)
    assert torch.equal(got, rope.apply(g, pos, grad=not grad))
    rope.apply(x, pos, grad=grad).sum().backward()
    assert torch.equal(x.grad, rope.apply(torch.ones_like(x), pos, grad=not grad))


def test_through_other_operations_and_by_differences():
    """d/dx of sum(w y^2), of which the rotation keeps nothing but its angle;
    and along a direction against differences: fp32 rounding of sums of 960
    terms of magnitude about 4, 2^-24 each, over a step of 2^-4 (2^-8 in all,
    relative to the sum of magnitudes)."""
    import moe_expert_ffn_dg_gb300 as pkg
    rope, pos = pkg.Rope(64), positions(5)
    gen = torch.Generator("cuda").manual_seed(3)
    x, w, e = (torch.randn(5, 3, 64, device="cuda", generator=gen) for _ in range(3))

    def loss(t):
        return (w * rope.apply(t, pos) ** 2).sum()
    x.requires_grad_()
    dx, = torch.autograd.grad(loss(x), x, create_graph=True)
    assert dx.requires_grad  # the gradient's own graph is there
    with torch.no_grad():
        step = 2.0 ** -4
        assert not rope.apply(x, pos).requires_grad
        diff = (loss(x + step * e).double() - loss(x - step * e).double()) / (2 * step)
        along = (dx.double() * e).sum()
        mag = (dx.abs() * e.abs()).sum()
        assert abs(diff - along) <= 2.0 ** -8 * mag


def test_a_given_output_records_nothing():
    import moe_expert_ffn_dg_gb300 as pkg
    rope, pos = pkg.Rope(64), positions(5)
    x = torch.randn(5, 3, 64, device="cuda", requires_grad=True)
    out = torch.empty(5, 3, 64, device="cuda")
    assert rope.apply(x, pos, out=out) is out and not out.requires_grad
    assert torch.equal(out, rope.apply(x, pos))


def test_backward_in_a_graph():
    """Forward and backward captured, while no eager graph of the leaf lives."""
    import moe_expert_ffn_dg_gb300 as pkg
    rope, pos = pkg.Rope(64), positions(5)
    x = torch.randn(5, 3, 64, device="cuda").to(BF).requires_grad_()
    g = torch.randn(5, 3, 64, device="cuda").to(BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(rope.apply(x, pos), x, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, = torch.autograd.grad(rope.apply(x, pos), x, g)
    g.copy_(torch.randn(5, 3, 64, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, rope.apply(g, pos, grad=True))
