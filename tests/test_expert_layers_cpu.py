"""The differentiable expert layer's front end, with a plain product in the place
of the library's: what needs no GPU."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import muon_step_03_amd as M
from muon_step_03_amd import layers


@pytest.fixture
def plain(monkeypatch):
    def forward(x, W, *, offsets):
        y = x.new_zeros(x.shape[0], W.shape[1])
        for e, (a, b) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
            y[a:b] = x[a:b] @ W[e].t()
        return y
    monkeypatch.setattr(layers, "linear_forward", forward)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("which", ["x", "W"])
def test_a_forward_mode_tangent_is_refused(plain, which, grad):
    """There is no forward-mode derivative: an output without a tangent would read
    as a derivative of zero."""
    x, W, o = torch.randn(6, 4), torch.randn(2, 3, 4), torch.tensor([0, 2, 5])
    with torch.set_grad_enabled(grad), fwd.dual_level():
        if which == "x":
            x = fwd.make_dual(x, torch.ones_like(x))
        else:
            W = fwd.make_dual(W, torch.ones_like(W))
        with pytest.raises(NotImplementedError):
            M.expert_linear(x, W, o)


def test_without_gradients(plain):
    x, W, o = torch.randn(6, 4), torch.randn(2, 3, 4), torch.tensor([0, 2, 5])
    want = layers.linear_forward(x, W, offsets=o)
    y = M.expert_linear(x, W, o)
    assert torch.equal(y, want) and not y.requires_grad
    for mode in (torch.no_grad(), torch.inference_mode()):
        with mode:      # nothing is kept: no checkpoint is made, which would need a GPU
            y = M.expert_linear(x, W.clone().requires_grad_(), o)
        assert torch.equal(y, want) and not y.requires_grad
