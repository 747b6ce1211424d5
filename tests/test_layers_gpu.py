"""The differentiable layers, and the optimizer steps on what they leave."""
import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from oracle import layer_oracle as lo

from _layers import DEV, check_backward, check_weight, f64, grads, hidden, params

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def leaf(t):
    return t.clone().requires_grad_()


@pytest.mark.parametrize("keep", [None, "e4m3", "int8"])
@pytest.mark.parametrize("bias", [True, False])
def test_layer_norm_gradients(keep, bias):
    x, dy = hidden(42, 136, BF16, seed=1), grads(42, 136, BF16, seed=1)
    g, b = params(136, F32)
    X, gain = leaf(x.view(6, 7, 136)), leaf(g)
    shift = leaf(b) if bias else None
    y = M.layer_norm(X, gain, shift, keep=keep)
    assert y.shape == X.shape
    direct = M.layernorm_forward(x, g, b if bias else None)
    assert torch.equal(y.view(42, 136), direct.y)
    y.backward(dy.view(6, 7, 136))
    seen = f64(x) if keep is None else lo.checkpoint(f64(x), keep)[0]
    check_backward((X.grad.view(42, 136), gain.grad, shift.grad if bias else None), dy, seen, g,
                   direct.mean, direct.rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keep", ["e4m3", "int8"])
def test_linear_gradients(dtype, keep):
    x, dz = hidden(42, 136, dtype, seed=2), grads(42, 72, dtype, seed=2)
    W = leaf(hidden(72, 136, dtype, seed=3, scale=0.05))
    X = leaf(x.view(2, 21, 136))
    z = M.linear(X, W, keep)
    assert torch.equal(z.detach(), X.detach() @ W.detach().t())
    z.backward(dz.view(2, 21, 72))
    assert W.grad.dtype == dtype
    check_weight(W.grad, dz, lo.checkpoint(f64(x), keep)[0])
    assert torch.equal(X.grad, dz.view(2, 21, 72) @ W.detach())


def test_gradients_against_differences():
    """The norm's and the weight's gradients of a float32 loss against central
    differences.  The input keeps its values in 8 bits exactly (multiples of
    1/8 up to 8 in int8), so the loss that is differentiated is the one that
    the kept input describes."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randint(-60, 61, (6, 32), generator=g) / 8.0).to(DEV)
    gain, bias = params(32, F32, seed=6)
    W = hidden(8, 32, F32, seed=7, scale=0.1)
    c, d = grads(6, 32, F32, seed=8) * 1e3, grads(6, 8, F32, seed=9) * 1e3

    def norm_loss(x, gain, bias):
        return float((lo.layernorm(f64(x), f64(gain), f64(bias), 1e-5)[0] * f64(c)).sum())

    X, G, B = leaf(x), leaf(gain), leaf(bias)
    (M.layer_norm(X, G, B, keep="int8") * c).sum().backward()
    h = 2.0 ** -8
    for grad, i in ((X.grad, 0), (G.grad, 1), (B.grad, 2)):
        base = [x, gain, bias]
        for at in list(np.ndindex(*grad.shape))[::7]:
            up, down = [t.clone() for t in base], [t.clone() for t in base]
            up[i][at] += h
            down[i][at] -= h
            span = float(up[i][at]) - float(down[i][at])
            slope = (norm_loss(*up) - norm_loss(*down)) / span
            # h^2 / 6 of a third derivative: the norm bends over its spread (about
            # 4 here), so under 1e-4 of the gradients' size of about 1 to 10
            assert abs(float(grad[at]) - slope) < 1e-3
    V = leaf(W)
    (M.linear(x, V, "int8") * d).sum().backward()
    want = f64(d).T @ f64(x)      # linear: its own difference quotient
    assert np.abs(f64(V.grad) - want).max() < 1e-5 * np.abs(f64(d)).sum() * 8


def test_shared_checkpoint_and_strided_gradients():
    """One checkpoint of the norm's output serves three projections; their
    gradients arrive as column slices of a fused one, and as an expanded one."""
    x, g = hidden(40, 96, BF16, seed=3), params(96, BF16)[0]
    Ws = [leaf(hidden(n, 96, BF16, seed=10 + n, scale=0.05)) for n in (32, 40, 56)]
    X, gain = leaf(x), leaf(g)
    y, ck = M.layer_norm(X, gain, keep="e4m3", y_keep="e4m3")
    z = torch.cat([M.linear(y, W, ck) for W in Ws], dim=1)
    dz = grads(40, 128, BF16, seed=4)
    z.backward(dz)
    y64 = lo.checkpoint(f64(y), "e4m3")[0]
    at = 0
    for W in Ws:
        n = W.shape[0]
        check_weight(W.grad, dz[:, at:at + n], y64)
        at += n
    assert bool(X.grad.isfinite().all()) and bool(gain.grad.isfinite().all())
    W = leaf(Ws[0].detach())
    M.linear(x, W).sum().backward()      # dy: ones, expanded with stride zero
    check_weight(W.grad, torch.ones(40, 32, dtype=BF16, device=DEV), lo.checkpoint(f64(x), "e4m3")[0])


def test_refusals():
    x, W = hidden(8, 64, BF16), hidden(16, 64, BF16, seed=1)
    ck = M.checkpoint_save(x[:5])
    with pytest.raises(ValueError, match="keep is"):
        M.linear(x, leaf(W), ck)
    with pytest.raises(ValueError, match="format"):
        M.linear(x, leaf(W), "fp4")
    with pytest.raises(ValueError, match="format"):
        M.layer_norm(x, leaf(x[0].contiguous()), keep="fp4")
    with torch.no_grad():      # nothing is kept, so nothing is asked of `keep`
        assert torch.equal(M.linear(x, W, ck), x @ W.t())
    X = leaf(x)
    (dx,) = torch.autograd.grad(M.layer_norm(X, x[0].contiguous()).float().square().sum(), X,
                                create_graph=True)
    with pytest.raises(RuntimeError):      # no second derivative
        dx.float().sum().backward()


def test_overwritten_checkpoint_is_noticed():
    x, W, gain = hidden(8, 64, BF16), leaf(hidden(16, 64, BF16, seed=1)), leaf(hidden(1, 64, BF16)[0])
    ck = M.checkpoint_save(x)
    for write in (lambda c: M.checkpoint_save(2 * x, out=c),
                  lambda c: M.layernorm_forward(x, gain.detach(), x_checkpoint=c)):
        z = M.linear(x, W, ck)
        write(ck)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.sum().backward()
    y, yc = M.layer_norm(x, gain, y_keep="int8")
    z = M.linear(y, W, yc)
    M.checkpoint_save(x, out=yc)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    kept = torch.empty(8, 64, dtype=BF16, device=DEV)
    y = M.layer_norm(kept.copy_(x), gain)
    M.checkpoint_restore(ck, out=kept)      # the norm's input, kept as it is
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        c = M.checkpoint_save(x)
        assert M.checkpoint_save(x, out=c) is c


def test_training_step_and_accumulated_micro_batches():
    """A small block trained by the hybrid optimizer, its hidden gradients
    formed once by autograd and once by accumulate_grad over micro-batches."""
    tokens, cols, rows = 256, 128, 192
    x = hidden(tokens, cols, BF16, seed=1)
    gain = torch.nn.Parameter(params(cols, F32)[0])
    W = torch.nn.Parameter(hidden(rows, cols, BF16, seed=2, scale=0.05))
    U = torch.nn.Parameter(hidden(cols, rows, BF16, seed=3, scale=0.05))
    opt = M.HybridMuonAdamW([W, U], [{"params": [gain], "lr": 0.015}])
    before = [p.detach().clone() for p in (W, U, gain)]
    for _ in range(2):
        for p in (W, U, gain):
            p.grad = None
        y, ck = M.layer_norm(x, gain, keep="int8", y_keep="e4m3")
        h = torch.relu(M.linear(y, W, ck))
        out = x + M.linear(h, U)
        (out.float() ** 2).mean().backward()
        opt.step()
    torch.cuda.synchronize()
    assert all(bool(p.isfinite().all()) and not torch.equal(p, b)
               for p, b in zip((W, U, gain), before))

    dz = grads(tokens, rows, BF16, seed=5)
    P = torch.nn.Parameter(hidden(rows, cols, F32, seed=6))
    step = M.MuonStep([P])
    kept = [M.checkpoint_save(x[a:a + 100], "int8") for a in (0, 100, 200)]
    for a, ck in zip((0, 100, 200), kept):
        step.accumulate_grad(0, dz[a:a + 100], ck)
    # three roundings of the running gradient on top of the sums
    x64 = np.concatenate([lo.checkpoint(f64(x[a:a + 100]), "int8")[0] for a in (0, 100, 200)])
    check_weight(P.grad, dz, x64, before=torch.zeros(rows, cols))
    with pytest.raises(ValueError, match="do not make"):
        step.accumulate_grad(0, dz[:, :8], kept[0])
    held = P.detach().clone()
    step.step()
    torch.cuda.synchronize()
    assert not torch.equal(P.detach(), held)


def test_captured_training_pass():
    """Forward and backward captured together and replayed on new inputs."""
    x = torch.empty(64, 128, dtype=BF16, device=DEV)
    gain = torch.nn.Parameter(params(128, BF16)[0])
    W = torch.nn.Parameter(hidden(96, 128, BF16, seed=2, scale=0.05))
    dz = grads(64, 96, BF16, seed=5)

    def run():
        y, ck = M.layer_norm(x, gain, keep="e4m3", y_keep="int8")
        return torch.autograd.grad(M.linear(y, W, ck), (W, gain), dz)

    x.copy_(hidden(64, 128, BF16, seed=0))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (1, 2, 3):
        x.copy_(hidden(64, 128, BF16, seed=seed))
        want = [t.clone() for t in run()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["transposed", "sliced", "columns"])
def test_linear_of_inputs_that_do_not_fold(dtype, layout):
    """Sequences read across, a slice of longer ones, columns outermost: the
    same values and gradients as of a contiguous copy."""
    base = hidden(84, 136, dtype, seed=2)
    x = {"transposed": base[:42].view(21, 2, 136).transpose(0, 1),
         "sliced": base.view(2, 42, 136)[:, 3:24],
         "columns": base[:42].t().contiguous().t().view(2, 21, 136)}[layout]
    assert not x.is_contiguous()
    W = hidden(72, 136, dtype, seed=3, scale=0.05)
    dz = grads(42, 72, dtype, seed=2).view(21, 2, 72).transpose(0, 1)
    got, want = [], []
    for a, b, to in ((x, dz, got), (x.contiguous(), dz.contiguous(), want)):
        X, V = a.detach().requires_grad_(), leaf(W)
        z = M.linear(X, V)
        to += [z.detach(), *torch.autograd.grad(z, (X, V), b)]
        z = M.linear(X, W)      # W frozen
        to += [z.detach(), *torch.autograd.grad(z, X, b)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    check_weight(got[2], dz.reshape(42, 72), lo.checkpoint(f64(x.reshape(42, 136)), "e4m3")[0])


@pytest.mark.parametrize("shape", [(0, 5, 64), (64,), (1, 64), (3, 1, 2, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layers_of_any_leading_dimensions(shape, dtype):
    """No token, one without a leading dimension, several dimensions."""
    x = hidden(max(1, int(np.prod(shape[:-1]))), 64, dtype, seed=1)[:int(np.prod(shape[:-1]))].view(shape)
    X, gain, bias = leaf(x), *(leaf(p) for p in params(64, dtype))
    W = leaf(hidden(24, 64, dtype, seed=3, scale=0.05))
    y, ck = M.layer_norm(X, gain, bias, keep="int8", y_keep="e4m3")
    z = M.linear(y, W, ck)
    assert y.shape == shape and z.shape == (*shape[:-1], 24) and ck.tokens == x.numel() // 64
    z.sum().backward()
    for t in (X, gain, bias, W):
        assert t.grad.shape == t.shape and bool(t.grad.isfinite().all())
    if x.numel():
        check_weight(W.grad, torch.ones(ck.tokens, 24, dtype=dtype, device=DEV),
                     lo.checkpoint(f64(y.view(-1, 64)), "e4m3")[0])
    else:
        assert not W.grad.any() and not gain.grad.any() and not bias.grad.any()


def test_shared_weights_broadcast_inputs_and_a_kept_graph():
    """A weight and a norm used twice, an input repeated along a batch, a graph
    run backward twice: gradients add up as PyTorch's do."""
    x = hidden(7, 64, F32, seed=1)
    X, gain, W = leaf(x), leaf(params(64, F32)[0]), leaf(hidden(64, 64, F32, seed=3, scale=0.05))
    wide = X.expand(5, 7, 64)
    z = M.linear(M.layer_norm(M.linear(M.layer_norm(wide, gain), W, "int8"), gain), W, "int8")
    dz = grads(35, 64, F32, seed=2).view(5, 7, 64)
    first = torch.autograd.grad(z, (X, gain, W), dz, retain_graph=True)
    again = torch.autograd.grad(z, (X, gain, W), dz)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # the same from separate leaves, added
    parts = [leaf(t.detach()) for t in (x.expand(5, 7, 64).contiguous(), gain, W, gain, W)]
    A, g1, W1, g2, W2 = parts
    z = M.linear(M.layer_norm(M.linear(M.layer_norm(A, g1), W1, "int8"), g2), W2, "int8")
    dA, dg1, dW1, dg2, dW2 = torch.autograd.grad(z, parts, dz)
    u = 2.0 ** -24
    for got, want, terms in ((first[0], dA.double().sum(0), dA.double().abs().sum(0)),
                             (first[1], dg1.double() + dg2.double(), dg1.abs().double() + dg2.abs().double()),
                             (first[2], dW1.double() + dW2.double(), dW1.abs().double() + dW2.abs().double())):
        # at most five additions in float32
        assert bool(((got.double() - want).abs() <= 5 * u * terms).all())
