"""The layer operators' fp64 definitions against independent facts (CPU):
finite differences, PyTorch's e4m3 conversion and the format's own limits."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo

RNG = np.random.default_rng(7)


def test_e4m3_numbers_and_ties():
    # the 126 finite magnitudes of e4m3 (PyTorch's decoding) are fixed points,
    # and halfway values go to the even neighbour
    mags = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lo.e4m3_round(mags), mags)
    mid = (mags[:-1] + mags[1:]) / 2
    even = mags[np.arange(126) + (np.arange(126) % 2)]
    assert np.array_equal(lo.e4m3_round(mid), even)
    v = RNG.uniform(-448, 448, 20000).astype(np.float32)
    v[:5000] *= np.float32(2.0) ** RNG.integers(-20, 0, 5000).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lo.e4m3_round(v.astype(np.float64)), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_checkpoint_scale_is_the_smallest_that_fits(fmt):
    top, e_min, e_max = lo.CKPT_FORMATS[fmt]
    x = RNG.standard_normal((50, 96)) * 10.0 ** RNG.integers(-20, 20, (50, 1))
    values, q, scale = lo.checkpoint(x, fmt)
    e = scale.astype(np.int64) - 127
    a = np.abs(x.reshape(50, 3, 32)).max(axis=2)
    assert np.all(a <= top * np.ldexp(1.0, e)) and np.all(a > top * np.ldexp(1.0, e - 1))
    # half a step: 2^-4 of the value (e4m3, or 2^-10 of the scale below its
    # normals), half of the scale (int8)
    s = np.ldexp(1.0, np.repeat(e, 32, axis=1))
    half = np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) if fmt == "e4m3" else s / 2
    assert np.all(np.abs(values - x) <= half)
    # every value is a bfloat16
    t = torch.from_numpy(values)
    assert torch.equal(t.to(torch.bfloat16).double(), t)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_checkpoint_borders(fmt):
    top, e_min, e_max = lo.CKPT_FORMATS[fmt]
    big = float(np.finfo(np.float32).max)
    x = np.zeros((6, 32))
    x[1, 3] = top
    x[2, 3] = top * 1.0000001
    x[3, 3] = big
    x[4, 3] = np.inf
    x[5, 3] = 2.0 ** -149
    values, q, scale = lo.checkpoint(x, fmt)
    assert scale[:, 0].tolist() == [10, 127, 128, e_max + 127, 255, 10]
    assert values[1, 3] == top and values[3, 3] == top * 2.0 ** e_max < big
    assert np.isnan(values[4]).all() and not q[4].any()
    assert not values[0].any() and not values[5].any()


def test_layernorm_gradients_against_differences():
    x, dy = RNG.standard_normal((5, 13)), RNG.standard_normal((5, 13))
    gain, bias = 1 + 0.1 * RNG.standard_normal(13), RNG.standard_normal(13)

    def loss(x, gain, bias):
        return (lo.layernorm(x, gain, bias, 1e-3)[0] * dy).sum()

    _, mean, rstd = lo.layernorm(x, gain, bias, 1e-3)
    dx, dgain, dbias = lo.layernorm_grad(dy, x, gain, mean, rstd)
    h = 1e-5

    def slope(i, at):
        args = [x, gain, bias]
        up, down = [a.copy() for a in args], [a.copy() for a in args]
        up[i][at] += h
        down[i][at] -= h
        return (loss(*up) - loss(*down)) / (2 * h)

    # central differences: error about h^2 of the third derivative plus
    # rounding 1e-16 / h
    for i, grad in enumerate((dx, dgain, dbias)):
        want = np.array([slope(i, at) for at in np.ndindex(grad.shape)]).reshape(grad.shape)
        assert np.abs(grad - want).max() < 1e-7


def test_weight_grad_groups():
    dy, x = RNG.standard_normal((9, 4)), RNG.standard_normal((9, 3))
    g = lo.weight_grad(dy, x, [0, 0, 5, 9])
    assert not g[0].any()
    assert np.allclose(g.sum(axis=0), lo.weight_grad(dy, x), atol=1e-12)
    w = RNG.standard_normal((4, 3))
    h = 1e-6
    e = np.zeros_like(w)
    e[2, 1] = h
    slope = (((x @ (w + e).T) * dy).sum() - ((x @ (w - e).T) * dy).sum()) / (2 * h)
    assert abs(lo.weight_grad(dy, x)[2, 1] - slope) < 1e-8
