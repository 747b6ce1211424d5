"""The layer operators at the ends of their types' ranges, against float64."""
import numpy as np
import pytest
import torch

import muon_step_03_amd as M

from _layers import DEV, check_weight, f64, hidden

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
