"""The differentiable layers whose products run in the library: ``expert_linear``,
and ``linear`` and ``expert_linear`` with products in 8 bits; and a mixture of
experts trained with them, Muon and AdamW with 8-bit states."""
import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from _linear import DEV, check, draw, f64, off, ragged
from _layers import check_weight
from oracle import layer_oracle as lo
from oracle import linear_oracle as lin

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def leaf(t):
    return t.clone().requires_grad_()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keep", ["e4m3", "int8"])
def test_expert_linear_gradients(dtype, keep):
    x, dz = draw(142, 136, dtype=dtype, seed=1), draw(142, 72, dtype=dtype, seed=2, scale=1e-2)
    o = ragged(142, 5, 3, before=4, behind=9)
    X, W = leaf(x), leaf(draw(5, 72, 136, dtype=dtype, seed=4, scale=0.1))
    z = M.expert_linear(X, W, off(o), keep)
    exact = dtype == BF16
    check(z, f64(x), f64(W), o, False, dtype, exact_products=exact)
    z.backward(dz)
    check(X.grad, f64(dz), f64(W), o, True, dtype, exact_products=exact)
    assert W.grad.dtype == dtype and W.grad.shape == W.shape
    check_weight(W.grad, dz, lo.checkpoint(f64(x), keep)[0], o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("given", [False, True])
def test_expert_linear_gradients_in_8_bits(dtype, given):
    x, dz = draw(300, 136, dtype=dtype, seed=1), draw(300, 200, dtype=dtype, seed=2, scale=1e-2)
    o = ragged(300, 5, 3, before=4, behind=9)
    w = draw(5, 200, 136, dtype=dtype, seed=4, scale=0.1)
    X, W = leaf(x), leaf(w)
    z = M.expert_linear(X, W, off(o), products=M.weight_quantize(w) if given else "e4m3")
    wv = np.stack([lin.quantized(m)[0] for m in f64(w)])
    xv, dv = lo.checkpoint(f64(x), "e4m3")[0], lo.checkpoint(f64(dz), "e4m3")[0]
    assert z.dtype == dtype
    check(z, xv, wv, o, False, dtype, eight=True)
    z.backward(dz)
    check(X.grad, dv, wv, o, True, dtype, eight=True)
    check_weight(W.grad, dz, xv, o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(6, 7, 136), (42, 136), (1, 136), (136,), (0, 136), (2, 0, 136)])
def test_linear_in_8_bits(dtype, shape):
    x = draw(*shape, dtype=dtype, seed=1)
    w = draw(200, 136, dtype=dtype, seed=4, scale=0.1)
    X, W = leaf(x), leaf(w)
    z = M.linear(X, W, products="e4m3")
    assert z.shape == (*shape[:-1], 200) and z.dtype == dtype
    dz = draw(*z.shape, dtype=dtype, seed=2, scale=1e-2)
    z.backward(dz)
    assert X.grad.shape == X.shape
    rows, wv = x.reshape(-1, 136), lin.quantized(f64(w))[0]
    xv, dv = lo.checkpoint(f64(rows), "e4m3")[0], lo.checkpoint(f64(dz.reshape(-1, 200)), "e4m3")[0]
    check(z.reshape(-1, 200), xv, wv, None, False, dtype, eight=True)
    check(X.grad.reshape(-1, 136), dv, wv, None, True, dtype, eight=True)
    check_weight(W.grad, dz.reshape(-1, 200), xv)
    with torch.no_grad():
        assert torch.equal(M.linear(x, w, products="e4m3"), z.detach())


def test_a_norms_checkpoint_feeds_the_product():
    """y's checkpoint from the norm is the product's operand: one rounding."""
    x, gain, w = draw(64, 256, seed=1), leaf(1 + draw(256, dtype=F32, scale=0.1)), leaf(draw(96, 256, scale=0.1))
    y, ck = M.layer_norm(leaf(x), gain, y_keep="e4m3")
    z = M.linear(y, w, ck, products="e4m3")
    want = M.linear_forward(ck, M.weight_quantize(w.detach()), dtype=BF16)
    assert torch.equal(z, want)
    z.sum().backward()
    assert gain.grad is not None and bool(torch.isfinite(gain.grad).all())


def test_gradients_against_differences():
    """A float32 loss, linear in each argument: its differences are its
    derivatives.  x and W hold few bits, so that their 8 bits are exact."""
    g = torch.Generator().manual_seed(5)
    ints = lambda *s: torch.randint(-7, 8, s, generator=g).float().to(DEV)  # noqa: E731
    x, W, r = ints(40, 32), ints(3, 24, 32), ints(40, 24)
    o = off([2, 17, 17, 36])
    for products in (None, "e4m3"):
        X, V = leaf(x), leaf(W)
        (M.expert_linear(X, V, o, products=products) * r).sum().backward()
        loss = lambda a, b: float((M.linear_forward(a, b, offsets=o).double() * r.double()).sum())  # noqa: E731
        base = loss(x, W)
        for t, e in ((3, 5), (20, 31), (0, 1), (39, 2), (35, 0)):
            a = x.clone()
            a[t, e] += 1
            assert loss(a, W) - base == float(X.grad[t, e])
        for e, i, j in ((0, 3, 4), (1, 0, 0), (2, 23, 31)):
            b = W.clone()
            b[e, i, j] += 1
            assert loss(x, b) - base == float(V.grad[e, i, j])


def test_what_is_asked_for_is_computed():
    x, w = draw(20, 64, seed=1), draw(2, 40, 64, seed=2)
    o = off([0, 5, 20])
    for products in (None, "e4m3"):
        X = leaf(x)
        M.expert_linear(X, w, o, products=products).sum().backward()     # no weight gradient
        assert X.grad is not None
        W = leaf(w)
        M.expert_linear(x, W, o, products=products).sum().backward()     # no input gradient
        assert W.grad is not None
    with torch.no_grad():
        z = M.expert_linear(leaf(x), leaf(w), o)
    assert not z.requires_grad and torch.equal(z, M.linear_forward(x, w, offsets=o))
    # expanded gradients and strided inputs
    X, W = leaf(draw(20, 128, seed=3)), leaf(w)
    z = M.expert_linear(X[:, 32:96], W, o)
    z.sum().backward()
    assert not X.grad[:, :32].any() and bool(X.grad[:, 32:96].any())
    # used twice, a graph kept: gradients add up
    X, W = leaf(x), leaf(w)
    z = M.expert_linear(X, W, o)
    z.sum().backward(retain_graph=True)
    one = W.grad.clone()
    z.sum().backward()
    assert torch.equal(W.grad, one + one)


def test_refusals():
    x, w, o = draw(20, 64), draw(2, 40, 64), off([0, 5, 20])
    for call, error in [
        (lambda: M.expert_linear(x[None], w, o), ValueError), (lambda: M.expert_linear(x, w[0], o), ValueError),
        (lambda: M.expert_linear(x.float(), w, o), TypeError), (lambda: M.expert_linear(x[:, :60], w, o), ValueError),
        (lambda: M.expert_linear(x, w, o[:2]), ValueError), (lambda: M.expert_linear(x, w, o.int()), TypeError),
        (lambda: M.expert_linear(x, w, None), ValueError),
        (lambda: M.linear(x, w[0], "int8", products="e4m3"), ValueError),
        (lambda: M.linear(x, w[0], M.checkpoint_save(x, "int8"), products="e4m3"), ValueError),
        (lambda: M.linear(x, w[0], M.checkpoint_save(x[:10]), products="e4m3"), ValueError),
        (lambda: M.linear(x, w[0], products="int8"), ValueError),
        (lambda: M.linear(x, w[0], products=M.weight_quantize(w)), ValueError),
    ]:
        with pytest.raises(error):
            call()


def test_an_overwritten_weight_is_noticed():
    x, w = draw(20, 64), leaf(draw(40, 64))
    w8 = M.weight_quantize(w.detach())
    z = M.linear(leaf(x), w, products=w8)
    M.weight_quantize(w.detach() * 2, out=w8)
    with pytest.raises(RuntimeError, match="modified"):
        z.sum().backward()


def loss_of(z2, y, order, top, head, products):
    out = torch.zeros_like(y).index_copy(0, order, z2) * top[:, None].to(BF16) + y
    return M.linear(out, head, products=products).float().square().mean()


@pytest.mark.parametrize("products", [None, "e4m3"])
def test_training_a_mixture_of_experts(products):
    """Norm, router, experts up and down, an output head: three steps with Muon on
    the experts (their gradient stacks as they come), AdamW with 8-bit states on
    the rest.  Every gradient is what autograd makes of plain products of the
    same 8-bit values, to bf16's roundings; the steps run and move the weights."""
    g = torch.Generator().manual_seed(11)
    T, C, H, E = 256, 128, 192, 6
    rnd = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(BF16).to(DEV)  # noqa: E731
    up = torch.nn.Parameter(rnd(E, H, C, scale=C ** -0.5))
    down = torch.nn.Parameter(rnd(E, C, H, scale=H ** -0.5))
    head = torch.nn.Parameter(rnd(64, C, scale=C ** -0.5))
    router = torch.nn.Parameter(rnd(E, C, scale=C ** -0.5))
    gain = torch.nn.Parameter(torch.ones(C, device=DEV, dtype=BF16))
    opt = M.AdamWStep([dict(params=[head, router], lr=1e-3), dict(params=[gain], lr=1e-3)], states="8bit")
    momenta = [torch.zeros(p.shape, dtype=F32, device=DEV) for p in (up, down)]
    for step in range(3):
        x = rnd(T, C)
        y, ck = M.layer_norm(x, gain, y_keep="e4m3")
        p = torch.softmax((y.detach() @ router.t()).float(), 1)
        top, e = p.max(1)
        order = torch.argsort(e, stable=True)
        o = torch.nn.functional.pad(torch.bincount(e, minlength=E).cumsum(0), (1, 0))
        z = y[order]
        w8 = [M.weight_quantize(w.detach()) for w in (up, down)] if products else [None, None]
        h = torch.relu(M.expert_linear(z, up, o, products=w8[0]))
        z2 = M.expert_linear(h, down, o, products=w8[1])
        loss = loss_of(z2, y, order, top, head, products)
        up.grad = down.grad = head.grad = router.grad = gain.grad = None
        loss.backward()
        before = [t.detach().clone() for t in (up, down, head, router, gain)]
        if step == 0:
            # the experts' gradients: autograd's, of plain float32 products of the values
            # that were multiplied (rounded to bf16 where the layers round)
            val = (lambda t: torch.from_numpy(lo.checkpoint(f64(t), "e4m3")[0]).float().to(DEV)) if products \
                else (lambda t: t.detach().float())
            wv = (lambda t: torch.from_numpy(np.stack([lin.quantized(m)[0] for m in f64(t)])).float().to(DEV)) \
                if products else (lambda t: t.detach().float())
            kept_z, kept_h = (torch.from_numpy(lo.checkpoint(f64(t), "e4m3")[0]).float().to(DEV) for t in (z, h))
            Z = leaf(z2.detach())
            dz2 = torch.autograd.grad(loss_of(Z, y.detach(), order, top.detach(), head, products), Z)[0]
            U, D = wv(up), wv(down)
            for k, (a, b) in enumerate(zip(o.tolist()[:-1], o.tolist()[1:])):
                if a == b:
                    assert not up.grad[k].any() and not down.grad[k].any()
                    continue
                gd = dz2[a:b].float().t() @ kept_h[a:b]
                dh = (val(dz2)[a:b] @ D[k]).to(BF16) * (h[a:b] > 0)
                gu = dh.float().t() @ kept_z[a:b]
                for got, want in ((down.grad[k], gd), (up.grad[k], gu)):
                    assert float((got.float() - want).norm()) <= 2.0 ** -6 * float(want.norm())
        with torch.no_grad():
            groups = [M.stacked_group(w.data, w.grad, m) for w, m in zip((up, down), momenta)]
            M.muon_step_grouped(groups, BF16, lr=0.01)
        opt.step()
        torch.cuda.synchronize()
        # the gain is 1 and its first step lr = 1e-3 at most: less than half of bf16's
        # spacing there, 2^-9 below 1, so that it rounds back; the others are small
        for t, b in zip((up, down, head, router, gain), before):
            assert bool(torch.isfinite(t).all())
            assert t is gain or not torch.equal(t.detach(), b)


@pytest.mark.parametrize("products", [None, "e4m3"])
def test_captured_training_pass(products):
    """Forward and backward of two expert layers in one graph, replayed with other
    values and other offsets between eager work: each replay's outputs and
    gradients are the eager ones."""
    x, W = draw(150, 64, seed=1), leaf(draw(4, 96, 64, seed=2, scale=0.1))
    V = leaf(draw(4, 64, 96, seed=3, scale=0.1))
    o = off(ragged(150, 4, 1, behind=3))

    def both():
        X = x.detach().requires_grad_()
        z = M.expert_linear(torch.relu(M.expert_linear(X, W, o, products=products)), V, o, products=products)
        return (z.detach(), *torch.autograd.grad(z, (X, W, V), torch.ones_like(z)))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in range(3):
        x.copy_(draw(150, 64, seed=10 + k))
        o.copy_(off(ragged(150, 4, 20 + k, behind=k)))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k
        del want


@pytest.mark.parametrize("products", [None, "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_that_are_not_contiguous(products, dtype):
    """Stacks kept with rows and columns exchanged, and slices of larger ones: the
    bits of a contiguous copy, and gradients in the parameter's own layout."""
    x, o = draw(50, 64, dtype=dtype, seed=1), off([3, 20, 20, 45])
    dz = draw(50, 40, dtype=dtype, seed=2)
    turned = leaf(draw(3, 64, 40, dtype=dtype, seed=3, scale=0.1))
    wide = leaf(draw(3, 40, 96, dtype=dtype, seed=4, scale=0.1))
    for p, view in ((turned, lambda t: t.transpose(1, 2)), (wide, lambda t: t[:, :, 16:80])):
        X, Y, W = leaf(x), leaf(x), leaf(view(p.detach()).contiguous())
        z, want = M.expert_linear(X, view(p), o, products=products), M.expert_linear(Y, W, o, products=products)
        assert torch.equal(z, want)
        z.backward(dz)
        want.backward(dz)
        assert torch.equal(X.grad, Y.grad) and torch.equal(view(p.grad), W.grad)
        with torch.no_grad():
            assert torch.equal(M.expert_linear(x, view(p), o, products=products), want)
    assert not wide.grad[:, :, :16].any() and not wide.grad[:, :, 80:].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens_and_an_expanded_gradient(dtype):
    """A batch without tokens whose outputs are summed: the gradient that autograd
    hands over is an expanded one of no elements, of any strides."""
    gain, w, W = leaf(draw(64, dtype=dtype)), leaf(draw(40, 64, dtype=dtype)), leaf(draw(2, 40, 64, dtype=dtype))
    o = off([0, 0, 0])
    for layer, p in ((lambda x: M.layer_norm(x, gain), gain), (lambda x: M.layer_norm(x, gain, keep="e4m3"), gain),
                     (lambda x: M.linear(x, w), w), (lambda x: M.linear(x, w, products="e4m3"), w),
                     (lambda x: M.expert_linear(x, W, o), W), (lambda x: M.expert_linear(x, W, o, products="e4m3"), W)):
        for shape in ((0, 64), (2, 0, 64)) if p is not W else ((0, 64),):
            x, p.grad = torch.zeros(shape, dtype=dtype, device=DEV, requires_grad=True), None
            layer(x).sum().backward()
            assert x.grad.shape == x.shape and p.grad.shape == p.shape and not p.grad.any()
    x = torch.zeros(1, 1, dtype=dtype, device=DEV).expand(0, 64)
    assert M.linear_forward(x, w.detach()).shape == (0, 40)
