"""Which matrix products the differentiable layers make (CPU).

Every product of ``linear`` is one of two matrices, whatever the strides of its
arguments: PyTorch turns x [a, b, cols] @ W^T whose leading dimensions do not fold
into a product over batches with W^T, a transposed view, as right operand of
each, which reads W once per batch and is not to be relied on in bfloat16.
"""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import muon_step_03_amd as M
from muon_step_03_amd import layers


class Products(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        name = func.overloadpacket.__name__
        if name in ("mm", "bmm", "baddbmm", "addmm", "mv"):
            self.made.append(name)
        return func(*args, **(kwargs or {}))


def arguments(layout):
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-4, 5, (2, 6, 16), generator=g).float()
    W = torch.randint(-4, 5, (8, 16), generator=g).float()
    if layout == "transposed":            # [sequence, batch] read as [batch, sequence]
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "sliced":
        x = torch.cat([x, x], dim=1)[:, :6]
    elif layout == "broadcast":
        x = x[:, :1].expand(2, 6, 16)
    elif layout == "columns":
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "none":
        x = x[:, :0]
    return x, W


LAYOUTS = ["contiguous", "transposed", "sliced", "broadcast", "columns", "none"]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_linear_without_a_weight_gradient(layout):
    x, W = arguments(layout)
    want = (x.reshape(-1, 16) @ W.t()).reshape(*x.shape[:2], 8)
    x.requires_grad_()
    with Products() as p:
        z = M.linear(x, W)
        (dx,) = torch.autograd.grad(z.sum(), x)      # dz: one element, expanded
    assert torch.equal(z, want) and torch.equal(dx, W.sum(0).expand(x.shape))
    assert p.made == ["mm", "mm"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dz", ["expanded", "transposed"])
def test_linear_with_one(layout, dz):
    """The two products of the layer's own function; the kept bytes play no part
    in them."""
    x, W = arguments(layout)
    want = (x.reshape(-1, 16) @ W.t()).reshape(*x.shape[:2], 8)
    x.requires_grad_()
    kept = torch.zeros(x.shape[0] * x.shape[1], 32, dtype=torch.int8)
    with Products() as p:
        z = layers._Linear.apply(x, W, kept, torch.zeros(kept.shape[0], 4, dtype=torch.uint8))
        d = torch.ones(1, 1, 1).expand(z.shape) if dz == "expanded" else \
            torch.ones(z.shape[1], z.shape[0], z.shape[2]).transpose(0, 1)
        (dx,) = torch.autograd.grad(z, x, d)
    assert torch.equal(z, want) and torch.equal(dx, W.sum(0).expand(x.shape))
    assert p.made == ["mm", "mm"]


def test_linear_of_one_token():
    x, W = arguments("contiguous")
    v = x[0, 0].clone().requires_grad_()
    z = M.linear(v, W)
    assert z.shape == (8,) and torch.equal(z, W @ v)
    (dx,) = torch.autograd.grad(z.sum(), v)
    assert torch.equal(dx, W.sum(0))
