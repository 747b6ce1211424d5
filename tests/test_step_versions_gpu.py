"""Steps tell autograd what they wrote: a backward pass that kept a weight which
was stepped since raises, as after PyTorch's own in-place steps."""
import pytest
import torch

import muon_step_03_amd as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _moments(p):
    return [torch.zeros(p.shape, dtype=F32, device=DEV) for _ in range(2)]


STEPS = {
    "adamw_step": lambda p: M.adamw_step(p, p.grad, *_moments(p), lr=0.01, step=1),
    "adamw8_step": lambda p: M.adamw8_step(p, p.grad, M.AdamwState8.zeros(p.numel(), DEV), lr=0.01, step=1),
    "AdamWStep": lambda p: M.AdamWStep([dict(params=[p], lr=0.01)]).step(),
    "AdamWStep 8bit": lambda p: M.AdamWStep([dict(params=[p], lr=0.01)], states="8bit").step(),
    "muon_step": lambda p: M.muon_step(p, p.grad, _moments(p)[0]),
    "muon_step_batched": lambda p: M.muon_step_batched([p], [p.grad], [_moments(p)[0]]),
    "MuonStep": lambda p: M.MuonStep([p]).step(),
    "HybridMuonAdamW": lambda p: M.HybridMuonAdamW([p], []).step(),
}


@pytest.mark.parametrize("name,experts", [(n, False) for n in STEPS] + [
    (n, True) for n in STEPS if n.lower().startswith("adamw")])      # Muon's have two dimensions
def test_a_stepped_weight_is_noticed(name, experts):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20, 64, generator=g).to(BF16).to(DEV).requires_grad_()
    shape = (2, 40, 64) if experts else (40, 64)
    W = torch.nn.Parameter((0.1 * torch.randn(shape, generator=g)).to(BF16).to(DEV))
    W.grad = torch.randn(shape, generator=g).to(BF16).to(DEV)
    o = torch.tensor([0, 7, 20], device=DEV)
    layer = (lambda: M.expert_linear(x, W, o)) if experts else (lambda: M.linear(x, W))
    z, before = layer(), W.detach().clone()
    STEPS[name](W)
    assert not torch.equal(W.detach(), before)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    assert x.grad is None
    layer().sum().backward()      # a pass that begins after the step goes through
    assert x.grad is not None


def test_what_a_step_writes_besides():
    P, G, m, v = (torch.rand(100, device=DEV) for _ in range(4))
    M.adamw_step(P, G, m, v, lr=0.01, step=1)
    assert [t._version for t in (P, G, m, v)] == [1, 0, 1, 1]
    st = M.AdamwState8.zeros(100, DEV)
    kept = st.m_q, st.m_scale, st.r_q, st.r_scale
    was = [t._version for t in kept]
    M.adamw8_step(P, G, st, lr=0.01, step=2)
    assert P._version == 2 and all(t._version > a for t, a in zip(kept, was))
    W, D, Q = (torch.rand(32, 64, device=DEV) for _ in range(3))
    M.muon_step(W, D, Q)
    assert [t._version for t in (W, D, Q)] == [1, 0, 1]


@pytest.mark.parametrize("name", ["AdamWStep", "AdamWStep 8bit", "MuonStep", "adamw_step", "adamw8_step"])
def test_tensors_without_a_version(name):
    with torch.inference_mode():
        p = torch.rand(32, 64, device=DEV)
        p.grad = torch.rand(32, 64, device=DEV)
        before = p.clone()
        STEPS[name](p)
        assert not torch.equal(p, before)
