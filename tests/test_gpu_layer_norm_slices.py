"""LayerNorm on tensors that start at any element, as slices and autograd's own gradients do."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import LayerNorm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _grads(x, w, b, gy):
    """LayerNorm's output and gradients on copies of their own, which start at 16 bytes."""
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, b)]
    y = LayerNorm.apply(*leaves, 1e-5)
    return y.detach(), *torch.autograd.grad(y, leaves, gy.clone())


@pytest.mark.parametrize("dt", list(ref.TYPES))
@pytest.mark.parametrize("cols", [7, 1411, 16391])
def test_gradient_of_a_joined_output(cols, dt):
    """The gradient of a part of torch.cat is a contiguous slice that starts at an odd element."""
    g = torch.Generator().manual_seed(cols)
    t = ref.TYPES[dt]
    a, b = (torch.randn(n, cols, generator=g).to(t).to(DEV) for n in (3, 5))
    w, s = (torch.randn(cols, generator=g).to(DEV) for _ in range(2))
    gy = torch.randn(8, cols, generator=g).to(t).to(DEV)
    leaves = [v.clone().requires_grad_() for v in (a, b, w, s)]
    y = torch.cat([LayerNorm.apply(leaves[0], leaves[2], leaves[3], 1e-5), LayerNorm.apply(leaves[1], leaves[2], leaves[3], 1e-5)])
    got = torch.autograd.grad(y, leaves, gy)
    first, second = _grads(a, w, s, gy[:3]), _grads(b, w, s, gy[3:])
    assert torch.equal(y, torch.cat([first[0], second[0]]))
    want = first[1], second[1], first[2] + second[2], first[3] + second[3]
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("dt", list(ref.TYPES))
@pytest.mark.parametrize("cols", [9, 40, 1411])
def test_slices_of_inputs_and_weights(cols, dt):
    """x from the second row on, weight and bias out of one flat tensor at an odd place, strides."""
    g = torch.Generator().manual_seed(cols)
    t = ref.TYPES[dt]
    x = torch.randn(6, cols, generator=g).to(t).to(DEV)
    flat = torch.randn(1 + 2 * cols, generator=g).to(DEV).requires_grad_()
    gy = torch.randn(5, cols, generator=g).to(t).to(DEV)
    leaf = x.clone().requires_grad_()
    w, b = flat[1:1 + cols], flat[1 + cols:]
    y = LayerNorm.apply(leaf[1:], w, b, 1e-5)
    gx, gf = torch.autograd.grad(y, (leaf, flat), gy)
    want = _grads(x[1:], w, b, gy)
    assert torch.equal(y, want[0]) and torch.equal(gx[1:], want[1]) and not gx[0].any()
    assert torch.equal(gf, torch.cat([gf.new_zeros(1), want[2], want[3]]))
    wide = torch.randn(cols, 2, generator=g).to(DEV)
    y = LayerNorm.apply(x.t().contiguous().t(), wide[:, 0], wide[:, 1], 1e-5)
    assert torch.equal(y, LayerNorm.apply(x, wide[:, 0].clone(), wide[:, 1].clone(), 1e-5))
