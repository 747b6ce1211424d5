"""C ABI checks of the linear products and of weights in 8 bits that need no GPU:
every call fails validation or has nothing to do, which precedes the first HIP
call.  The oracle is pinned by PyTorch's e4m3."""
import ctypes
import os

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib
from oracle import linear_oracle as lin

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmuon.so not built")
F32, BF16 = _lib.MUON_DTYPE_F32, _lib.MUON_DTYPE_BF16
A = [0x100000000 * (i + 1) for i in range(12)]
OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
BIG = _lib.MUON_MAX_DIM


def plain(fn, x=A[0], ld=None, dtype=BF16, W=A[1], offsets=A[2], count=4, tokens=16, rows=32, cols=64,
          y=A[3]):
    ld = (cols if fn == "forward" else rows) if ld is None else ld
    call = getattr(_lib.lib(), "muon_linear_" + fn)
    return call(x, ld, dtype, W, offsets, count, tokens, rows, cols, y, None)


@built
@pytest.mark.parametrize("fn", ["forward", "input_grad"])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(x=None), ARG), (dict(W=None), ARG), (dict(y=None), ARG),
    (dict(offsets=None), ARG), (dict(count=-1), ARG), (dict(count=0, offsets=None), ARG),
    (dict(count=1025), SHAPE), (dict(rows=0), SHAPE), (dict(cols=BIG + 1), SHAPE), (dict(rows=BIG + 1), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(tokens=_lib.MUON_MAX_TOKENS + 1), SHAPE),
    (dict(x=A[0] + 1), ARG), (dict(W=A[1] + 2, dtype=F32), ARG), (dict(y=A[3] + 1), ARG), (dict(offsets=A[2] + 4), ARG),
    (dict(ld=31), ARG), (dict(ld=(1 << 24) + 1), ARG),
    (dict(y=A[0]), ARG), (dict(y=A[1] + 4 * 32 * 64 * 2 - 2), ARG), (dict(y=A[2] - 2), ARG), (dict(y=A[2] + 38), ARG),
    # more tiles than a launch has blocks
    (dict(tokens=1 << 30, rows=BIG, cols=BIG, x=1 << 48, y=1 << 50), SHAPE),
])
def test_product_refusals(fn, kw, status):
    assert plain(fn, **kw) == status


@built
def test_products_of_nothing():
    for fn in ("forward", "input_grad"):
        assert plain(fn, tokens=0, x=None, W=None, y=None) == OK
        assert plain(fn, tokens=0, count=0, x=None, W=None, y=None) == OK


def weight(q=A[4], q_t=A[5], scale=A[6], count=4, rows=32, cols=64):
    return ctypes.byref(_lib.Weight8(q, q_t, scale, count, rows, cols))


def ckpt(tokens=16, cols=64, fmt=0, q=A[0], scale=A[1]):
    return ctypes.byref(_lib.Ckpt(q, scale, tokens, cols, fmt))


def quantized(fn, ck=None, w=None, offsets=A[2], y=A[3], dtype=BF16):
    call = getattr(_lib.lib(), f"muon_linear_{fn}_quantized")
    ck = ckpt(cols=64 if fn == "forward" else 32) if ck is None else ck
    return call(ck, weight() if w is None else w, offsets, y, dtype, None)


WEIGHT_FAULTS = [(dict(q=None), ARG), (dict(q_t=None), ARG), (dict(scale=None), ARG), (dict(q=A[4] + 8), ARG),
                 (dict(q_t=A[5] + 1), ARG), (dict(count=-1), SHAPE), (dict(count=1025), SHAPE),
                 (dict(rows=0), SHAPE), (dict(cols=BIG + 1), SHAPE)]


@built
@pytest.mark.parametrize("kw,status", WEIGHT_FAULTS)
def test_weight_descriptor(kw, status):
    assert _lib.lib().muon_weight_quantize(A[0], BF16, weight(**kw), None) == status
    for fn in ("forward", "input_grad"):
        assert quantized(fn, w=weight(**kw)) == status


@built
def test_quantize_refusals():
    q = _lib.lib().muon_weight_quantize
    assert q(A[0], 9, weight(), None) == DTYPE
    assert q(A[0], BF16, None, None) == ARG
    assert q(None, BF16, weight(), None) == ARG
    assert q(A[0] + 1, BF16, weight(), None) == ARG
    assert q(A[4], BF16, weight(), None) == ARG                       # W over q
    assert q(A[6] - 2, BF16, weight(), None) == ARG                   # W over the scales
    assert q(A[0], BF16, weight(q_t=A[4] + 4 * 32 * 128 - 16), None) == ARG
    assert q(None, BF16, weight(count=0, q=None, q_t=None, scale=None), None) == OK
    # 2^24 blocks
    w = weight(A[4], 0x7000000000000, 0x7f00000000000, 1024, 128 * 128, 128 * 128)
    assert q(0x10000000000, F32, w, None) in (ARG, SHAPE)


@built
@pytest.mark.parametrize("fn,inner", [("forward", 64), ("input_grad", 32)])
def test_quantized_product_refusals(fn, inner):
    assert quantized(fn, dtype=4) == DTYPE
    assert quantized(fn, ck=ckpt(cols=inner + 1)) == SHAPE
    assert quantized(fn, ck=ckpt(cols=inner, fmt=1)) == ARG           # int8
    assert quantized(fn, ck=ckpt(cols=inner, fmt=2)) == ARG
    assert quantized(fn, ck=ckpt(cols=inner, q=None)) == ARG
    assert quantized(fn, offsets=None) == ARG
    assert quantized(fn, y=None) == ARG
    assert quantized(fn, y=A[5]) == ARG
    assert quantized(fn, y=A[6] + 2) == ARG
    assert quantized(fn, ck=ckpt(tokens=0, cols=inner, q=None, scale=None), y=None) == OK
    call = getattr(_lib.lib(), f"muon_linear_{fn}_quantized")
    assert call(None, weight(), A[2], A[3], BF16, None) == ARG
    assert call(ckpt(cols=inner), None, A[2], A[3], BF16, None) == ARG


def test_front_end_without_a_gpu():
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="GPU"):
        M.linear_forward(x, W)
    with pytest.raises(TypeError):
        M.linear_forward(None, W)
    with pytest.raises(TypeError):
        M.linear_input_grad([1.0], W)
    with pytest.raises(ValueError, match="GPU"):
        M.weight_quantize(W)
    with pytest.raises(ValueError, match="GPU"):
        M.Weight8.empty(6, 8, device="cpu")


def test_oracle_of_weights_matches_torch():
    g = torch.Generator().manual_seed(0)
    W = 0.02 * torch.randn(200, 300, generator=g)
    values, q, scale = lin.quantized(W.double().numpy())
    for i in range(2):
        for j in range(3):
            b = W[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            s = float(scale[i, j]) - 127
            assert 224 < float(b.abs().max()) / 2 ** s <= 448
            want = (b * 2.0 ** -s).to(torch.float8_e4m3fn).double().numpy()
            assert np.array_equal(q[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128], want)
            assert np.array_equal(values[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128], want * 2.0 ** s)


def test_oracle_of_ragged_products():
    g = np.random.default_rng(0)
    x, W = g.standard_normal((9, 4)), g.standard_normal((3, 5, 4))
    y = lin.forward(x, W, [1, 4, 3, 12])
    assert not y[0].any()
    assert np.allclose(y[1:4], x[1:4] @ W[0].T) and np.allclose(y[4:], x[4:] @ W[2].T)
    assert np.allclose(lin.input_grad(y, W, [1, 4, 3, 12])[5], y[5] @ W[2])
    assert lin.bounds([-3, 100, 5], 9).tolist() == [0, 9, 9]


@built
def test_kernel_choice_refuses_what_calls_refuse():
    k = _lib.lib().muon_linear_kernel
    assert k(0, 0, 1, 1, 4096, 1024, BF16) == _lib.MUON_LINEAR_FEW
    assert k(1, 0, 64, 49152, 1408, 512, BF16) in range(5)
    for bad in ((0, 0, 0, 1, 64, 64, 0), (0, 0, 1025, 1, 64, 64, 0), (0, 0, 1, 0, 64, 64, 0),
                (0, 0, 1, 1, 0, 64, 0), (0, 0, 1, 1, 64, BIG + 1, 0), (0, 0, 1, 1, 64, 64, 2),
                (0, 0, 1, 1 << 30, BIG, BIG, 0)):
        assert k(*bad) == -1


def test_grids_of_short_rows_count_their_smaller_tiles():
    """Rows shorter than 16 bytes are computed in tiles of 64 whatever the choice
    for longer ones is: four times the blocks."""
    k = _lib.lib().muon_linear_kernel
    tokens = 1 << 24
    assert k(0, 0, 1, tokens, 4096, 8, BF16) == _lib.MUON_LINEAR_TILES_128
    assert k(0, 0, 1, tokens, 4096, 7, BF16) == -1
    assert k(1, 0, 1, tokens, 7, 4096, BF16) == -1
    assert k(0, 0, 1, tokens // 2, 4096, 7, BF16) >= 0


@built
@pytest.mark.parametrize("across,rows,cols,dtype", [
    (0, 4096, 5, BF16), (0, 4096, 7, BF16), (0, 4096, 3, F32), (1, 5, 4096, BF16), (1, 4096, 7, BF16),
    (1, 3, 4096, F32), (1, 4096, 2, F32)])
def test_short_rows_are_reported_in_the_tiles_that_they_take(across, rows, cols, dtype):
    """Rows of operands below 16 bytes always take tiles of 64 (or the kernel for
    few tokens), those of outputs alone do not."""
    k = _lib.lib().muon_linear_kernel
    for tokens in (300, 5000, 16384, 200_000):
        assert k(across, 0, 1, tokens, rows, cols, dtype) == _lib.MUON_LINEAR_TILES_64
    assert k(0, 0, 1, 1, 40, 5, BF16) == _lib.MUON_LINEAR_FEW
    assert k(0, 0, 1, 1 << 20, 5, 64, BF16) == _lib.MUON_LINEAR_TILES_128


@built
@pytest.mark.parametrize("across", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("count", [1, 37, 1024])
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 4096), (4096, 7), (64, 64), (65, 1), (1, 65), (513, 300), (BIG, 64), (64, BIG)])
def test_the_largest_call_is_the_documented_one(across, dtype, count, rows, cols):
    """Sizes are refused from (tokens / S + count + 2) * ceil(n / S) >= 2^24 - 8 on,
    S the side of the tiles that muon_linear_kernel names."""
    k = _lib.lib().muon_linear_kernel
    n = cols if across else rows
    for tokens in [1 << i for i in range(31)] + [3 << i for i in range(28)]:
        which = k(across, 0, count, tokens, rows, cols, dtype)
        sides = {_lib.MUON_LINEAR_FEW: 16, _lib.MUON_LINEAR_TILES_64: 64}
        if which >= 0:
            s = sides.get(which, 128)
            assert (tokens // s + count + 2) * -(-n // s) < (1 << 24) - 8
        else:       # (tiles of 128 are fewer than those of 64)
            assert (tokens // 64 + count + 2) * -(-n // 64) >= (1 << 24) - 8
    # what fits a GPU's memory in tiles of 64 without part tiles is taken
    assert k(0, 0, 1, (1 << 24) - 1024, 4096, 1024, BF16) >= 0
    assert k(across, 0, 1, (1 << 30) - (1 << 20), 1, 1, dtype) == _lib.MUON_LINEAR_TILES_64
    assert k(across, 0, 1, 1 << 30, 1, 1, dtype) == -1


@built
def test_the_largest_weight():
    """2^24 blocks of 128 x 128 are refused, with no overlap that could refuse them."""
    w = weight(A[4], 0x7000000000000, 0x7f00000000000, 1024, 128 * 128, 128 * 128)
    assert _lib.lib().muon_weight_quantize(0x10000000000, F32, w, None) == SHAPE


@pytest.mark.parametrize("field", ["q", "q_t", "scale", "shape", "device"])
def test_a_weights_fields_are_not_assigned(field):
    """The library reads the tensors, and the sizes, that a weight was made of."""
    with pytest.raises(AttributeError):
        setattr(object.__new__(M.Weight8), field, None)
