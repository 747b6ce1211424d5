"""Optimizer steps are launched on their parameters' device, whichever is current:
shown with stand-ins for the parameters and the grouped calls, on no GPU."""
import contextlib
import types

import pytest
import torch

from muon_step_03_amd import api


@pytest.fixture
def current(monkeypatch):
    now = [torch.device("cuda", 0)]

    @contextlib.contextmanager
    def device(d):
        was, now[0] = now[0], torch.device(d)
        yield
        now[0] = was
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "_wrote", lambda *t: None)
    return now


def parameter(device, dtype):
    p = types.SimpleNamespace(device=torch.device(device), dtype=dtype, grad=object())
    p.data = p
    return p


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_adamw(monkeypatch, current, states):
    calls = []
    for name in ("adamw", "adamw8"):
        monkeypatch.setattr(api, name + "_tensor", lambda p, *a, **kw: p)
        monkeypatch.setattr(api, name + "_step_grouped",
                            lambda t, dtype, **kw: calls.append((current[0], dtype, t)))
    opt = object.__new__(api.AdamWStep)
    opt.betas, opt.eps, opt.seed, opt.step_count = (0.8, 0.95), 1e-8, 0, 0
    params = [parameter(d, t) for t in (torch.float32, torch.bfloat16) for d in ("cuda:1", "cuda:0", "cuda:1")]
    opt.entries = [(p, None, None, 0.1, 0.0) for p in params]
    opt.states = None if states == "f32" else [None] * len(params)
    opt.step()
    assert sum(len(t) for _, _, t in calls) == len(params) and len(calls) == 4
    for device, dtype, tensors in calls:
        assert all(p.device == device and p.dtype == dtype for p in tensors)
    assert current[0] == torch.device("cuda", 0)


def test_muon(monkeypatch, current):
    calls = []
    monkeypatch.setattr(api, "workspace_bytes_grouped", lambda *a: 0)
    monkeypatch.setattr(api, "muon_step_grouped",
                        lambda g, dtype, device, **kw: calls.append((current[0], device)))
    opt = object.__new__(api.MuonStep)
    opt.params, opt.hp = [parameter("cuda:1", torch.float32)], {}
    opt._by_dtype = {torch.float32: {(4, 4): [0]}}
    opt._workspaces = {torch.float32: types.SimpleNamespace(device=torch.device("cuda:1"), numel=lambda: 1)}
    opt._groups = lambda dtype, shapes: ([], [])
    opt.step()
    assert calls == [(torch.device("cuda:1"),) * 2]
