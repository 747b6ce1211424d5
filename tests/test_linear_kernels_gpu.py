"""Each kernel of the linear products at the sizes that it is chosen for, asserted,
against products in float64 on the GPU (bounds of ``_linear``)."""
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib
from _linear import DEV, HALF, U, off, ragged

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FEW, T64, T128, S128, S256 = range(5)


def kernel(across, eight, count, tokens, rows, cols, dtype):
    return _lib.lib().muon_linear_kernel(int(across), int(eight), count, tokens, rows, cols,
                                         _lib.MUON_DTYPE_BF16 if dtype == BF16 else _lib.MUON_DTYPE_F32)


def draw(*shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(*shape, generator=g, device=DEV)
    x.view(-1)[::97] *= 8.0
    return x.to(dtype)


def close(y, x, W, offsets, across, eight):
    """y against x W^T (or x W) in float64, matrix by matrix; x and W float64."""
    k = x.shape[1]
    ends = [0, x.shape[0]] if offsets is None else offsets
    live = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        live[a:b] = True
        if a == b:
            continue
        B = (W if offsets is None else W[e])
        B = B if across else B.t()
        for i in range(a, b, 4096):
            j = min(i + 4096, b)
            want, mag = x[i:j] @ B, x[i:j].abs() @ B.abs()
            bound = (k + 9) * U * mag
            if eight and y.dtype == BF16:
                big = sum(x[i:j, c:c + 64].abs().amax(1, keepdim=True) * B[c:c + 64].abs().amax(0, keepdim=True)
                          for c in range(0, k, 64))
                bound = bound + 64 * 2.0 ** -13 * big
                err = (y[i:j].double() - want).norm()
                assert float(err) <= (2.0 ** -8 + 2.0 ** -13) * float(want.norm())
            bound = bound + HALF[y.dtype] * (want.abs() + bound)
            assert float(((y[i:j].double() - want).abs() - bound).max()) <= 0, (e, i)
    assert not bool(y[~live].any())


CASES = [  # which, across, eight bits, count, tokens, rows, cols, type of the result
    (FEW, False, False, 1, 16, 4096, 1024, BF16), (FEW, False, False, 40, 64, 130, 333, BF16),
    (FEW, False, False, 6, 90, 777, 1001, F32), (FEW, False, True, 1, 1, 5632, 2048, BF16),
    (FEW, True, True, 5, 40, 777, 1411, F32), (FEW, False, False, 3, 20, 50, 5, BF16),
    (FEW, False, False, 3, 20, 50, 3, F32), (FEW, False, False, 4, 30, 100, 30, BF16),
    (T64, False, False, 7, 1000, 513, 200, BF16), (T64, True, False, 7, 500, 1001, 777, BF16),
    (T64, True, False, 5, 300, 1001, 333, F32), (T64, False, True, 4, 700, 640, 777, F32),
    (T64, True, False, 3, 100, 5, 77, BF16), (T64, True, False, 3, 100, 77, 5, BF16),
    (T64, True, False, 3, 100, 3, 2, F32), (T64, False, True, 6, 900, 500, 130, BF16),
    (T128, False, False, 4, 5000, 1000, 96, BF16), (T128, True, False, 4, 5000, 96, 1001, BF16),
    (T128, False, False, 1, 8200, 1030, 77, F32), (T128, True, False, 1, 8200, 64, 1028, F32),
    (T128, False, True, 4, 5000, 1000, 200, BF16), (T128, True, True, 3, 5000, 333, 1000, F32),
    (S128, False, False, 5, 6000, 1416, 64, BF16), (S128, False, False, 70, 9000, 1024, 192, BF16),
    (S128, False, False, 1, 4100, 2056, 128, BF16), (S128, False, True, 5, 6000, 1416, 128, BF16),
    (S128, False, True, 1, 8000, 1288, 384, BF16), (S128, True, True, 3, 7000, 256, 1416, BF16),
    (S256, False, False, 3, 5000, 6144, 1024, BF16), (S256, True, False, 1, 4000, 4096, 4096, BF16),
    (S256, False, True, 3, 5000, 6144, 1024, BF16), (S256, True, True, 1, 4096, 4096, 4096, BF16),
    (S256, False, False, 1, 4090, 4088, 2048, BF16),
]


@pytest.mark.parametrize("which,across,eight,count,tokens,rows,cols,dtype", CASES)
def test_kernel(which, across, eight, count, tokens, rows, cols, dtype):
    assert kernel(across, eight, count, tokens, rows, cols, dtype) == which
    shape = (rows, cols) if count == 1 else (count, rows, cols)
    W = draw(*shape, dtype=F32 if eight else dtype, seed=1) / 16
    W = W.to(W.dtype if eight else dtype)
    x = draw(tokens, rows if across else cols, dtype=F32 if eight else dtype, seed=2)
    o = None if count == 1 else ragged(tokens, count, 3, before=tokens // 50, behind=tokens // 40)
    fn = M.linear_input_grad if across else M.linear_forward
    if eight:
        ck, w8 = M.checkpoint_save(x, "e4m3"), M.weight_quantize(W)
        y = fn(ck, w8, offsets=off(o), dtype=dtype)
        xv = M.checkpoint_restore(ck, F32).double()
        s = torch.exp2(w8.scale.double() - 127).repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)
        wv = (w8.q.double() * s)[..., :cols]
    else:
        y = fn(x, W, offsets=off(o))
        xv, wv = x.double(), W.double()
    close(y, xv, wv, o, across, eight)


@pytest.mark.parametrize("which,tokens,rows,cols", [(S128, 25_700, 32768, 64), (S256, 49_500, 32768, 576)])
def test_more_tiles_per_block_than_the_table_holds(which, tokens, rows, cols):
    """Over 96 tiles of each block: its table of places is refilled under way."""
    assert kernel(False, False, 3, tokens, rows, cols, BF16) == which
    W, x = draw(3, rows, cols, dtype=BF16, seed=4), draw(tokens, cols, dtype=BF16, seed=5)
    o = [0, tokens // 3, tokens // 3 + 1000, tokens - 300]
    y = M.linear_forward(x, W, offsets=off(o))
    assert not bool(y[tokens - 300:].any())
    g = torch.Generator(device=DEV).manual_seed(6)
    for e, (a, b) in enumerate(zip(o[:-1], o[1:])):
        pick = torch.randint(a, b, (200,), generator=g, device=DEV)
        pick[0], pick[1] = a, b - 1
        want, mag = x[pick].double() @ W[e].double().t(), x[pick].double().abs() @ W[e].double().abs().t()
        bound = (cols + 9) * U * mag
        bound = bound + HALF[BF16] * (want.abs() + bound)
        assert float(((y[pick].double() - want).abs() - bound).max()) <= 0
    # every row was written: none is all zeros
    assert bool((y[:tokens - 300].abs().amax(1) > 0).all())


def test_unaligned_rows_take_other_tiles():
    """Sizes of the blocks that stay, rows that do not start on 16 bytes."""
    for across in (False, True):
        rows, cols, tokens = 4096, 4096, 4000
        assert kernel(across, False, 1, tokens, rows, cols, BF16) in (S128, S256)
        W = draw(rows, cols, dtype=BF16, seed=1)
        wide = draw(tokens, 4099, dtype=BF16, seed=2)
        fn = M.linear_input_grad if across else M.linear_forward
        close(fn(wide[:, 3:], W), wide[:, 3:].double(), W.double(), None, across, False)


def test_two_streams_at_once():
    """Calls that overlap on two streams share nothing."""
    W, x = draw(3, 4096, 1024, dtype=BF16, seed=1), draw(5000, 1024, dtype=BF16, seed=2)
    W2, x2 = draw(64, 512, 1408, dtype=BF16, seed=3), draw(48, 1408, dtype=BF16, seed=4)
    o, o2 = off(ragged(5000, 3, 1)), off(ragged(48, 64, 2))
    want, want2 = M.linear_forward(x, W, offsets=o), M.linear_forward(x2, W2, offsets=o2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(M.linear_forward(x, W, offsets=o, stream=a), M.linear_forward(x2, W2, offsets=o2, stream=b))
           for _ in range(4)]
    torch.cuda.synchronize()
    for y, y2 in got:
        assert torch.equal(y, want) and torch.equal(y2, want2)


def test_more_than_2_to_the_32_outputs():
    """131073 tokens of 32768 outputs: rows past 2^32 elements are theirs."""
    tokens, rows, cols = 131_073, 32768, 64
    W, x = draw(rows, cols, dtype=BF16, seed=7), draw(tokens, cols, dtype=BF16, seed=8)
    y = M.linear_forward(x, W)
    for pick in (torch.arange(0, 130, device=DEV), torch.arange(tokens - 130, tokens, device=DEV)):
        want, mag = x[pick].double() @ W.double().t(), x[pick].double().abs() @ W.double().abs().t()
        bound = (cols + 9) * U * mag
        bound = bound + HALF[BF16] * (want.abs() + bound)
        assert float(((y[pick].double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("which,across,tokens,rows,cols", [(S128, False, 4100, 2048, 128), (S256, False, 4000, 4096, 4096),
                                                           (T128, True, 8200, 64, 1024)])
@pytest.mark.parametrize("at", [8, 5])
def test_outputs_that_begin_inside_a_line(which, across, tokens, rows, cols, at):
    """Lines of 128 bytes are stored past the L2, parts of lines through it: the same
    bits, and what lies before and behind stays as it was."""
    assert kernel(across, False, 1, tokens, rows, cols, BF16) == which
    W, x = draw(rows, cols, dtype=BF16, seed=1), draw(tokens, rows if across else cols, dtype=BF16, seed=2)
    fn = M.linear_input_grad if across else M.linear_forward
    want = fn(x, W)
    buf = torch.full((want.numel() + 64,), 7.0, dtype=BF16, device=DEV)
    out = buf[at:at + want.numel()].view(want.shape)
    assert torch.equal(fn(x, W, out=out), want)
    assert bool((buf[:at] == 7).all()) and bool((buf[at + want.numel():] == 7).all())
