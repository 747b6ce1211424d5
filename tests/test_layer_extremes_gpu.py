"""The layer operators at the ends of their types' ranges, against float64."""
import numpy as np
import pytest
import torch

import muon_step_03_amd as M

from _layers import (DEV, HALF, ROW, U, check_backward, check_weight, f64, grads, hidden, params,
                     within)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# a few tokens, and a size that the 256 x 256 tiles take
SIZES = [(40, 24, 64), (640, 4096, 2056)]


@pytest.mark.parametrize("tokens,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt,byte", [("e4m3", 246), ("int8", 248)])
def test_weight_grad_of_the_largest_activations(tokens, rows, cols, dtype, fmt, byte):
    """Blocks at the largest scale, up to the largest finite value, with dy so
    small that every sum stays finite."""
    x = (hidden(tokens, cols, F32, seed=1).clamp(-1, 1).double() * torch.finfo(dtype).max).to(dtype)
    dy = hidden(tokens, rows, dtype, seed=2, scale=1e-6)
    dy[:, 0] = 0.0
    ck = M.checkpoint_save(x, fmt)
    assert int(ck.scale.max()) == byte
    x64 = f64(M.checkpoint_restore(ck, F32))
    assert np.isfinite(x64).all()
    for gdtype in (BF16, F32):
        G = M.weight_grad(dy, ck, dtype=gdtype)
        assert not G[0].any()
        check_weight(G, dy, x64)


@pytest.mark.parametrize("exponent", [-100, -108, -112, -120, -128, -136, -146])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", SIZES)
def test_weight_grad_of_tiny_gradients(tokens, rows, cols, dtype, exponent):
    """dy down to subnormal numbers against activations so large that G is not.
    float32 dy may lose half of bf16's smallest step, 2^-134, per element."""
    g = torch.Generator().manual_seed(-exponent)
    x = (torch.randint(-127, 128, (tokens, cols), generator=g) * 2.0 ** 90).to(dtype).to(DEV)
    dy = torch.randn(tokens, rows, generator=g, dtype=torch.float64) * 2.0 ** exponent
    dy = dy.to(dtype).to(DEV)
    x64, d64 = f64(x), f64(dy)
    ck = M.checkpoint_save(x, "int8")
    assert np.array_equal(f64(M.checkpoint_restore(ck, F32)), x64)
    want = d64.T @ x64
    parts, lost = (1, 0.0) if dtype == BF16 else (3, 2.0 ** -134)
    bound = (parts * tokens + 4) * U * (np.abs(d64).T @ np.abs(x64)) + lost * np.abs(x64).sum(0)
    for gdtype in (BF16, F32):
        within(M.weight_grad(dy, ck, dtype=gdtype), want,
               bound + HALF[gdtype] * (np.abs(want) + bound), "G")


@pytest.mark.parametrize("cols", [7, 200, 777, 2304, 8200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layernorm_rows_beyond_float32(cols, dtype):
    """Rows whose sum or squares leave float32 give what the formula gives in
    float32: an infinite sum an infinite mean, infinite squares rstd = 0."""
    x = hidden(9, cols, dtype, seed=cols)
    gain, bias = params(cols, dtype)
    clean = M.layernorm_forward(x, gain, bias)
    x[1] = (hidden(1, cols, F32, seed=9)[0].double() * 1e25).to(dtype)    # squares
    x[2] = 3e38                                                           # the sum
    x[3] = -3e38
    inf = float("inf")
    x[4, 5] = inf
    x[5, 5] = -inf
    x[6, 2], x[6, 5] = inf, -inf
    out = M.layernorm_forward(x, gain, bias, y_checkpoint="e4m3")
    whole = [0, 7, 8]
    for a, b in zip(out[:3], clean[:3]):
        assert torch.equal(a[whole], b[whole])
    x64 = f64(x[1])
    within(out.mean[1:2], x64.mean(keepdims=True), (ROW + 3 * U) * np.abs(x64).mean(), "mean")
    assert out.rstd[1] == 0 and torch.equal(out.y[1], bias)
    assert out.mean[2:6].tolist() == [inf, -inf, inf, -inf] and out.mean[6].isnan()
    # centred at an infinity: (-inf)^2 = inf, rstd = 0; inf - inf = NaN
    assert not out.rstd[2:4].any() and out.rstd[4:7].isnan().all() and out.y[2:7].isnan().all()
    assert (out.y_checkpoint.scale[2:7, :-(-cols // 32)] == 255).all()
    assert (out.y_checkpoint.scale[[0, 1, 7, 8]] != 255).all()


@pytest.mark.parametrize("cols", [7, 200, 777, 2304, 8200])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [6, 3000])
def test_layernorm_backward_rows_beyond_float32(cols, dtype, tokens):
    """A row with rstd = 0 gives dx = 0 and nothing to dgain; an infinite dy
    leaves infinities, and NaN only where two of them meet."""
    if tokens * cols > 2 ** 22:
        tokens = 600
    x, dy = hidden(tokens, cols, dtype, seed=1), grads(tokens, cols, dtype, seed=1)
    x[2] = (hidden(1, cols, F32, seed=9)[0].double() * 1e25).to(dtype)
    gain, bias = params(cols, dtype)
    out = M.layernorm_forward(x, gain, bias)
    got = M.layernorm_backward(dy, x, gain, out.mean, out.rstd)
    assert not got[0][2].any()
    check_backward(got, dy, f64(x), gain, out.mean, out.rstd)
    dy[4, 5] = float("inf")
    got = M.layernorm_backward(dy, x, gain, out.mean, out.rstd)
    assert got[0][4].isinf().any()
    with np.errstate(invalid="ignore"):
        check_backward(got, dy, f64(x), gain, out.mean, out.rstd)
