"""The layer operators on the GPU against their float64 definitions."""
import copy
import pickle

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib
from oracle import layer_oracle as lo

from _layers import (DEV, check_backward, check_checkpoint, check_forward, check_weight, f64,
                     grads, hidden, params)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FMTS = ["e4m3", "int8"]


# ------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,cols", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 100), (64, 768),
                                         (33, 777), (130, 1408), (2, 32768), (257, 129)])
def test_checkpoint(tokens, cols, dtype, fmt):
    x = hidden(tokens, cols, dtype, seed=cols)
    ck = M.checkpoint_save(x, fmt)
    values = check_checkpoint(ck, f64(x), fmt)
    for out in (BF16, F32):
        assert np.array_equal(f64(M.checkpoint_restore(ck, out)), values)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_checkpoint_borders(dtype, fmt):
    top = lo.CKPT_FORMATS[fmt][0]
    big = torch.finfo(dtype).max
    x = torch.zeros(12, 96)
    x[1, 3], x[1, 40] = top, -top * 2.0 ** 30
    x[2, 3], x[2, 70] = top * (1 + 2.0 ** -7), top * (1 - 2.0 ** -7)
    x[3, 0], x[3, 95] = big, -big
    x[4, 5], x[4, 6] = float("inf"), 1.0
    x[5, 64], x[5, 65] = float("nan"), 1.0
    x[6, 31], x[6, 32] = 2.0 ** -126, -2.0 ** -133        # subnormal in both types
    x[7] = torch.arange(96) - 48.0                        # every half-way value of small integers
    x[8] = (torch.arange(96) - 48.0) * 2.0 ** -120
    x[9, 0], x[9, 1:32] = 2.0 ** 100, 1.0                 # one outlier in a block
    x[10] = -0.0
    x[11, :32] = torch.linspace(1, 2, 32)
    x = x.to(dtype).to(DEV)
    ck = M.checkpoint_save(x, fmt)
    values = check_checkpoint(ck, f64(x), fmt)
    got = f64(M.checkpoint_restore(ck, F32))
    assert np.array_equal(got, values, equal_nan=True)
    assert np.isnan(got[4, :32]).all() and not np.isnan(got[4, 32:]).any()


def test_checkpoint_strided_odd_start_and_out():
    wide = hidden(40, 500, BF16, seed=3)
    x = wide[3:, 11:312]                      # row stride 500, starts at an odd element
    out = M.ActCheckpoint.empty(37, 301, "int8", DEV)
    out.q.fill_(99)
    out.scale.fill_(99)
    assert M.checkpoint_save(x, out=out) is out
    values = check_checkpoint(out, f64(x), "int8")
    into = torch.full((37, 301), 7.0, dtype=F32, device=DEV)
    assert M.checkpoint_restore(out, out=into) is into
    assert np.array_equal(f64(into), values)


@pytest.mark.parametrize("dtype,cols", [(BF16, 2000), (F32, 1000), (F32, 1001)])
def test_checkpoint_larger_than_the_caches(dtype, cols):
    x = hidden(500, cols, dtype).repeat(80, 1)      # over 2^27 bytes
    assert x.numel() * x.element_size() > 2 ** 27
    ck = M.checkpoint_save(x, "int8")
    near = M.checkpoint_restore(M.checkpoint_save(x[:500], "int8"), dtype)
    assert torch.equal(M.checkpoint_restore(ck, dtype).view(80, 500, cols),
                       near.expand(80, 500, cols))


def test_checkpoint_no_tokens():
    ck = M.checkpoint_save(torch.empty(0, 70, dtype=BF16, device=DEV))
    assert ck.shape == (0, 70) and M.checkpoint_restore(ck).shape == (0, 70)


# --------------------------------------------------------------- layer norm
SHAPES = [(1, 1), (1, 768), (3, 31), (5, 512), (9, 513), (64, 768), (33, 777), (130, 1024),
          (17, 1408), (6, 2048), (5, 2049), (7, 4096), (3, 5632), (2, 8192), (3, 8193),
          (2, 20000), (2, 32768)]


@pytest.mark.parametrize("tokens,cols", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layernorm(tokens, cols, dtype, pdtype):
    x, dy = hidden(tokens, cols, dtype, seed=cols), grads(tokens, cols, dtype, seed=cols)
    gain, bias = params(cols, pdtype)
    out = M.layernorm_forward(x, gain, bias, eps=1e-5)
    check_forward(out, x, gain, bias, 1e-5)
    assert out.x_checkpoint is None and out.y_checkpoint is None
    got = M.layernorm_backward(dy, x, gain, out.mean, out.rstd)
    check_backward(got, dy, f64(x), gain, out.mean, out.rstd)


@pytest.mark.parametrize("tokens,cols", [(1, 40), (33, 777), (65, 1024), (4, 2049), (3, 8193)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("xf,yf", [("e4m3", "int8"), ("int8", "e4m3"), (None, "e4m3"), ("e4m3", None)])
def test_layernorm_through_checkpoints(tokens, cols, dtype, xf, yf):
    x, dy = hidden(tokens, cols, dtype, seed=cols), grads(tokens, cols, dtype, seed=cols)
    gain, bias = params(cols, dtype)
    out = M.layernorm_forward(x, gain, None, x_checkpoint=xf, y_checkpoint=yf)
    check_forward(out, x, gain, None, 1e-5)
    if yf:   # of y as returned, bit for bit
        check_checkpoint(out.y_checkpoint, f64(out.y), yf)
    if xf:
        kept = check_checkpoint(out.x_checkpoint, f64(x), xf)
        dx, dgain, dbias = M.layernorm_backward(dy, out.x_checkpoint, gain, out.mean, out.rstd,
                                                bias=False)
        assert dbias is None
        check_backward((dx, dgain, None), dy, kept, gain, out.mean, out.rstd)


@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("tokens", [1, 8, 9, 5000])
def test_layernorm_backward_accumulates(tokens, dtype, pdtype):
    cols = 200
    x, dy = hidden(tokens, cols, dtype, seed=5), grads(tokens, cols, dtype, seed=5)
    gain, bias = params(cols, pdtype)
    out = M.layernorm_forward(x, gain, bias)
    dgain, dbias = params(cols, pdtype, seed=9)
    before = (dgain.clone(), dbias.clone())
    got = M.layernorm_backward(dy, x, gain, out.mean, out.rstd, dgain=dgain, dbias=dbias,
                               accumulate=True)
    assert got[1] is dgain and got[2] is dbias
    check_backward(got, dy, f64(x), gain, out.mean, out.rstd, before)


def test_layernorm_strided_views():
    wide, dwide = hidden(50, 900, BF16, seed=4), grads(50, 901, BF16, seed=4)
    x, dy = wide[1:, 101:402], dwide[:49, 7:308]
    gain, bias = params(301, F32)
    out = M.layernorm_forward(x, gain, bias, x_checkpoint="e4m3")
    check_forward(out, x, gain, bias, 1e-5)
    check_backward(M.layernorm_backward(dy, x, gain, out.mean, out.rstd), dy, f64(x), gain,
                   out.mean, out.rstd)


def test_layernorm_no_tokens():
    gain, bias = params(64, F32)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    out = M.layernorm_forward(x, gain, bias, y_checkpoint="int8")
    assert out.y.shape == (0, 64) and out.mean.shape == (0,)
    dx, dgain, dbias = M.layernorm_backward(x, x, gain, out.mean, out.rstd)
    assert dx.shape == (0, 64) and not dgain.any() and not dbias.any()
    before = torch.ones_like(gain)
    M.layernorm_backward(x, x, gain, out.mean, out.rstd, dgain=before, dbias=dbias, accumulate=True)
    assert bool((before == 1).all())


def test_layernorm_large_offset_and_bad_rows():
    """A mean 1000 times the spread; rows with an infinity or a NaN leave the
    others as they are."""
    x = hidden(9, 600, F32, seed=8) + 1000.0
    gain, bias = params(600, F32)
    check_forward(M.layernorm_forward(x, gain, bias), x, gain, bias, 1e-5)
    clean = M.layernorm_forward(x, gain, bias, y_checkpoint="e4m3")
    x[2, 7], x[5, 599] = float("inf"), float("nan")
    out = M.layernorm_forward(x, gain, bias, y_checkpoint="e4m3")
    keep = torch.tensor([0, 1, 3, 4, 6, 7, 8], device=DEV)
    assert torch.equal(out.y[keep], clean.y[keep])
    assert torch.equal(out.y_checkpoint.q[keep].view(torch.uint8),
                       clean.y_checkpoint.q[keep].view(torch.uint8))
    assert bool(out.y[[2, 5]].isnan().all()) and bool((out.y_checkpoint.scale[[2, 5], :19] == 255).all())


# --------------------------------------------------------- weight gradients
def weight_case(tokens, rows, cols, dtype, fmt, seed=0):
    dy = grads(tokens, rows, dtype, seed)
    ck = M.checkpoint_save(hidden(tokens, cols, dtype, seed), fmt)
    return dy, ck, f64(M.checkpoint_restore(ck, F32))


@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 128, 128), (31, 64, 96), (32, 128, 128), (33, 129, 127), (96, 768, 768),
    (127, 257, 33), (500, 100, 1000), (1024, 512, 1408), (2049, 333, 257), (5000, 130, 70),
    (4096, 256, 512), (65, 1024, 40)])
@pytest.mark.parametrize("dtype,gdtype,fmt", [(BF16, BF16, "e4m3"), (BF16, F32, "int8"),
                                              (F32, F32, "e4m3"), (F32, BF16, "int8")])
def test_weight_grad(tokens, rows, cols, dtype, gdtype, fmt):
    dy, ck, x64 = weight_case(tokens, rows, cols, dtype, fmt, seed=rows)
    G = M.weight_grad(dy, ck, dtype=gdtype)
    assert G.dtype == gdtype
    check_weight(G, dy, x64)
    before = params(rows * cols, gdtype, seed=3)[0].view(rows, cols)
    into = before.clone()
    assert M.weight_grad(dy, ck, G=into, accumulate=True) is into
    check_weight(into, dy, x64, before=before)


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64)


@pytest.mark.parametrize("counts", [
    [0], [0, 0, 0], [5], [0, 7, 0, 0, 300, 1], [32] * 5, [1] * 70, [900, 0, 3, 2100, 31, 33],
    [0] * 64 + [500] + [0] * 64 + [700]])
@pytest.mark.parametrize("dtype,fmt", [(BF16, "e4m3"), (BF16, "int8"), (F32, "int8")])
def test_weight_grad_ragged(counts, dtype, fmt):
    rows, cols = 136, 200
    tokens = sum(counts) + 9      # tokens that belong to nobody
    dy, ck, x64 = weight_case(tokens, rows, cols, dtype, fmt, seed=len(counts))
    off = offsets_of(counts)
    G = M.weight_grad(dy, ck, offsets=off.to(DEV))
    check_weight(G, dy, x64, off.tolist())
    empty = [i for i, c in enumerate(counts) if c == 0]
    assert not G[empty].any()
    before = torch.randn(G.shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV) * 1e-2
    into = before.clone()
    M.weight_grad(dy, ck, offsets=off.to(DEV), G=into, accumulate=True)
    assert torch.equal(into[empty], before[empty])
    check_weight(into, dy, x64, off.tolist(), before)


# Sizes whose work takes the 256 x 256 tiles: whole and odd rows (repacked),
# columns that end inside a tile, steps of 32 tokens that do not come out even.
WIDE = [(4100, 1001, 1030), (8201, 520, 264), (33000, 256, 8), (2817, 1408, 512), (32800, 8, 100)]


@pytest.mark.parametrize("tokens,rows,cols", WIDE)
@pytest.mark.parametrize("dtype,gdtype,fmt", [(BF16, BF16, "int8"), (BF16, F32, "e4m3"),
                                              (F32, F32, "int8"), (F32, BF16, "e4m3")])
def test_weight_grad_wide(tokens, rows, cols, dtype, gdtype, fmt):
    dy, ck, x64 = weight_case(tokens, rows, cols, dtype, fmt, seed=rows)
    check_weight(M.weight_grad(dy, ck, dtype=gdtype), dy, x64)


@pytest.mark.parametrize("counts", [
    [0, 1, 31, 32, 33, 2000, 64, 0, 3839], [7000], [0, 6500, 0], [96] * 70, [3001, 3001],
    [1] * 900 + [6200] + [0] * 300])
@pytest.mark.parametrize("dtype,rows,fmt", [(BF16, 512, "e4m3"), (BF16, 517, "int8"), (F32, 512, "int8")])
def test_weight_grad_wide_ragged(counts, dtype, rows, fmt):
    cols = 520
    if len(counts) > 64:
        rows, cols = (rows + 7) // 8, 72      # many small matrices
    tokens = sum(counts) + 3
    dy, ck, x64 = weight_case(tokens, rows, cols, dtype, fmt, seed=len(counts))
    off = offsets_of(counts)
    before = torch.randn(len(counts), rows, cols, generator=torch.Generator().manual_seed(1))
    before = before.to(dtype).to(DEV) * 1e-2
    into = before.clone()
    M.weight_grad(dy, ck, offsets=off.to(DEV), G=into, accumulate=True)
    check_weight(into, dy, x64, off.tolist(), before)
    check_weight(M.weight_grad(dy, ck, offsets=off.to(DEV)), dy, x64, off.tolist())


@pytest.mark.parametrize("bad,read_as", [
    ([-50, 3000, 9000, 10 ** 12], [0, 3000, 8000, 8000]),
    ([0, 8000, 0, 8000, 0, 8000], [0, 8000, 8000, 8000, 8000, 8000]),
])
def test_weight_grad_wide_bad_offsets(bad, read_as):
    dy, ck, x64 = weight_case(8000, 512, 260, BF16, "int8")
    G = M.weight_grad(dy, ck, offsets=torch.tensor(bad, dtype=torch.int64, device=DEV))
    check_weight(G, dy, x64, read_as)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(8192, 512, 512), (5003, 700, 300), (5003, 701, 300)])
def test_weight_grad_wide_exact_integers(dtype, tokens, rows, cols):
    g = torch.Generator().manual_seed(tokens + rows)
    x = torch.randint(-1, 2, (tokens, cols), generator=g).float()
    lim = 128 if dtype == BF16 else 1900
    dy = torch.randint(-lim, lim + 1, (tokens, rows), generator=g).float()
    want = dy.double().t() @ x.double()
    assert float(want.abs().max()) < 2 ** 24
    dy = dy.to(dtype).to(DEV)
    for fmt in FMTS:
        ck = M.checkpoint_save(x.to(dtype).to(DEV), fmt)
        assert torch.equal(M.weight_grad(dy, ck, dtype=F32).cpu().double(), want)
    # a strided view: its own row stride, 16-byte rows or (from an odd column) not
    wide = torch.full((tokens, rows + 24), float("nan"), dtype=dtype, device=DEV)
    for start in (8, 3):
        view = wide[:, start:start + rows]
        view.copy_(dy)
        assert torch.equal(M.weight_grad(view, ck, dtype=F32).cpu().double(), want)
        wide.fill_(float("nan"))


@pytest.mark.parametrize("dtype,rows", [(BF16, 512), (BF16, 500), (BF16, 501), (F32, 256)])
def test_weight_grad_wide_keeps_bad_tokens_apart(dtype, rows):
    """NaN and infinities of one matrix's tokens, and of its neighbours' in the
    same steps, stay out of the others."""
    tokens, cols = 9000, 512
    dy, x = grads(tokens, rows, dtype, seed=6), hidden(tokens, cols, dtype, seed=6)
    off = torch.tensor([0, 3001, 3002, 9000], dtype=torch.int64, device=DEV)
    clean = M.weight_grad(dy, M.checkpoint_save(x, "int8"), offsets=off)
    dy[3001, :] = float("nan")
    x[3001, 40] = float("inf")
    for fmt in FMTS:
        ck = M.checkpoint_save(x, fmt)
        got = M.weight_grad(dy, ck, offsets=off)
        assert bool(got[1].isnan().all()) and not bool(got[[0, 2]].isnan().any())
        if fmt == "int8":
            assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    dy[3001, :] = 1.0
    dy[3001, 5] = float("inf")
    x[3001, 40] = 2.0
    x[3001, 64:96] = float("inf")      # a marked block
    x[3001, 96:128] = 3.0
    for fmt in FMTS:
        got = M.weight_grad(dy, M.checkpoint_save(x, fmt), offsets=off)
        assert bool(got[1][:, 64:96].isnan().all()) and not bool(got[[0, 2]].isnan().any())
        assert bool((got[1][5, 96:128] == float("inf")).all())
        assert bool(got[1][torch.arange(rows) != 5][:, 96:128].isfinite().all())


def test_weight_grad_offsets_start_late():
    dy, ck, x64 = weight_case(300, 64, 64, BF16, "e4m3")
    off = torch.tensor([17, 100, 100, 260], dtype=torch.int64)
    check_weight(M.weight_grad(dy, ck, offsets=off.to(DEV)), dy, x64, off.tolist())
    assert M.weight_grad(dy, ck, offsets=off[:1].to(DEV)).shape == (0, 64, 64)


@pytest.mark.parametrize("bad,read_as", [
    ([-50, 100, 400, 10 ** 12], [0, 100, 300, 300]),
    ([0, 200, 100, 300], [0, 200, 200, 300]),
    ([0, 300, 0, 300, 0, 300], [0, 300, 300, 300, 300, 300]),
    ([-2 ** 62, 2 ** 62, -2 ** 62, 2 ** 62], [0, 300, 300, 300]),
])
def test_weight_grad_bad_offsets_are_bounded(bad, read_as):
    dy, ck, x64 = weight_case(300, 64, 64, BF16, "int8")
    G = M.weight_grad(dy, ck, offsets=torch.tensor(bad, dtype=torch.int64, device=DEV))
    check_weight(G, dy, x64, read_as)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(700, 192, 320), (3000, 300, 130), (64, 512, 256)])
def test_weight_grad_exact_integers(dtype, tokens, rows, cols):
    """Integer inputs whose sums stay under 2^24 come out exactly: every index,
    and the three parts of a float32 dy, in one equality."""
    g = torch.Generator().manual_seed(tokens)
    x = torch.randint(-1, 2, (tokens, cols), generator=g).float()
    lim = 128 if dtype == BF16 else 5000
    dy = torch.randint(-lim, lim + 1, (tokens, rows), generator=g).float()
    ck = M.checkpoint_save(x.to(dtype).to(DEV), "int8")
    G = M.weight_grad(dy.to(dtype).to(DEV), ck, dtype=F32)
    want = dy.double().t() @ x.double()
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(G.cpu().double(), want)


def test_weight_grad_strided_and_other_tokens():
    """dy a column slice of a fused gradient at an odd element; NaN in the
    tokens of one matrix stays out of the others'."""
    wide = grads(400, 700, BF16, seed=6)
    dy = wide[:, 13:213]
    ck = M.checkpoint_save(hidden(400, 96, BF16, seed=6), "e4m3")
    x64 = f64(M.checkpoint_restore(ck, F32))
    check_weight(M.weight_grad(dy, ck, dtype=F32), dy, x64)
    off = torch.tensor([0, 150, 151, 400], dtype=torch.int64, device=DEV)
    clean = M.weight_grad(dy, ck, offsets=off)
    wide[150, :] = float("nan")
    got = M.weight_grad(dy, ck, offsets=off)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    assert bool(got[1].isnan().all())
    x = hidden(400, 96, BF16, seed=6)
    x[150, 40] = float("inf")
    got = M.weight_grad(grads(400, 200, BF16), M.checkpoint_save(x, "int8"), offsets=off)
    assert bool(got[1][:, 32:64].isnan().all()) and not bool(got[[0, 2]].isnan().any())
    assert not bool(got[1][:, :32].isnan().any()) and not bool(got[1][:, 64:].isnan().any())


def test_weight_grad_float32_infinity():
    dy = torch.zeros(40, 8, dtype=F32, device=DEV)
    dy[3, 2], dy[5, 4] = float("inf"), torch.finfo(F32).max
    x = torch.ones(40, 8, dtype=F32, device=DEV)
    G = M.weight_grad(dy, M.checkpoint_save(x, "e4m3"))
    assert bool((G[2] == float("inf")).all())
    assert bool((G[4] == torch.finfo(F32).max).all())
    assert not bool(G[[0, 1, 3, 5, 6, 7]].any())


# Sizes whose estimated times choose the 256 x 256 tiles: whole rows, and odd
# ones, which are repacked; matrices in one part and in several.
LARGE = [(640, 4096, 2056), (2100, 2056, 2050), (2100, 2051, 2050), (5003, 2056, 1030)]


@pytest.mark.parametrize("tokens,rows,cols", LARGE)
@pytest.mark.parametrize("gdtype,fmt", [(BF16, "int8"), (F32, "e4m3")])
def test_weight_grad_large(tokens, rows, cols, gdtype, fmt):
    dy, ck, x64 = weight_case(tokens, rows, cols, BF16, fmt, seed=rows)
    into = params(rows * cols, gdtype, seed=3)[0].view(rows, cols)
    before = into.clone()
    check_weight(M.weight_grad(dy, ck, dtype=gdtype), dy, x64)
    check_weight(M.weight_grad(dy, ck, G=into, accumulate=True), dy, x64, before=before)


COUNTS = [0, 1, 31, 32, 33, 2000, 64, 0, 3839, 1000, 700, 1300]


@pytest.mark.parametrize("rows", [776, 771])
@pytest.mark.parametrize("fmt", FMTS)
def test_weight_grad_large_ragged(rows, fmt):
    dy, ck, x64 = weight_case(9003, rows, 1030, BF16, fmt, seed=rows)
    off = offsets_of(COUNTS)
    G = M.weight_grad(dy, ck, offsets=off.to(DEV))
    check_weight(G, dy, x64, off.tolist())
    assert not G[[0, 7]].any()
    before = torch.randn(G.shape, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV) * 1e-2
    into = before.clone()
    M.weight_grad(dy, ck, offsets=off.to(DEV), G=into, accumulate=True)
    check_weight(into, dy, x64, off.tolist(), before)
    # tokens of one matrix that are NaN, in steps that its neighbours share
    dy[off[5] - 1] = float("nan")
    again = M.weight_grad(dy, ck, offsets=off.to(DEV))
    assert bool(again[4].isnan().all())
    others = [i for i in range(12) if i != 4]
    assert torch.equal(again[others], G[others])
    bad = torch.tensor([-7, 0, 10 ** 12] + [5] * 9 + [-1], dtype=torch.int64, device=DEV)
    dy[off[5] - 1] = 0.0
    got = M.weight_grad(dy, ck, offsets=bad)
    check_weight(got[1:2], dy, x64, [0, 9003])
    assert not got[[0, *range(2, 12)]].any()


@pytest.mark.parametrize("rows", [2056, 2051])
def test_weight_grad_large_exact_integers(rows):
    tokens, cols = 2100, 2050
    g = torch.Generator().manual_seed(rows)
    x = torch.randint(-1, 2, (tokens, cols), generator=g).to(BF16).to(DEV)
    dy = torch.randint(-128, 129, (tokens, rows), generator=g).to(BF16).to(DEV)
    want = dy.cpu().double().t() @ x.cpu().double()
    wide = torch.full((tokens, rows + 24), float("nan"), dtype=BF16, device=DEV)
    for fmt in FMTS:
        ck = M.checkpoint_save(x, fmt)
        assert torch.equal(M.weight_grad(dy, ck, dtype=F32).cpu().double(), want)
        for start in (8, 3):      # rows that start on 16 bytes, and rows that do not
            view = wide[:, start:start + rows]
            view.copy_(dy)
            assert torch.equal(M.weight_grad(view, ck, dtype=F32).cpu().double(), want)
            wide.fill_(float("nan"))


# Rows that end inside a vector, before its end, or with it.
@pytest.mark.parametrize("cols", [2, 3, 5, 6, 7, 9, 11, 12, 15, 250, 509, 1027])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_row_ends(cols, dtype):
    tokens = 37
    x, dy = hidden(tokens, cols, dtype, seed=cols), grads(tokens, cols, dtype, seed=cols)
    gain, bias = params(cols, dtype)
    out = M.layernorm_forward(x, gain, bias, x_checkpoint="int8", y_checkpoint="e4m3")
    check_forward(out, x, gain, bias, 1e-5)
    check_checkpoint(out.x_checkpoint, f64(x), "int8")
    check_checkpoint(out.y_checkpoint, f64(out.y), "e4m3")
    check_backward(M.layernorm_backward(dy, x, gain, out.mean, out.rstd), dy, f64(x), gain,
                   out.mean, out.rstd)
    check_weight(M.weight_grad(dy, out.x_checkpoint), dy, f64(M.checkpoint_restore(out.x_checkpoint, F32)))
    # the same rows with others' bytes on both sides: nothing of them gets in
    w = torch.full((tokens, cols + 9), float("nan"), dtype=dtype, device=DEV)
    dw = w.clone()
    w[:, 4:4 + cols], dw[:, 5:5 + cols] = x, dy
    at = M.layernorm_forward(w[:, 4:4 + cols], gain, bias, x_checkpoint="int8")
    assert torch.equal(at.y, out.y) and torch.equal(at.x_checkpoint.q, out.x_checkpoint.q)
    for a, b in zip(M.layernorm_backward(dw[:, 5:5 + cols], w[:, 4:4 + cols], gain, out.mean, out.rstd),
                    M.layernorm_backward(dy, x, gain, out.mean, out.rstd)):
        assert torch.equal(a, b)
    assert torch.equal(M.weight_grad(dw[:, 5:5 + cols], out.x_checkpoint),
                       M.weight_grad(dy, out.x_checkpoint))


# ----------------------------------------------------- how calls are made
def test_same_bits_every_time_and_given_buffers():
    x, dy = hidden(3000, 520, BF16, seed=2), grads(3000, 520, BF16, seed=2)
    gain, bias = params(520, F32)
    out = M.layernorm_forward(x, gain, bias, y_checkpoint="e4m3")
    first = M.layernorm_backward(dy, x, gain, out.mean, out.rstd)
    G = M.weight_grad(dy, out.y_checkpoint)
    ws = torch.full((max(M.layernorm_workspace_bytes(3000, 520),
                         M.weight_grad_workspace_bytes(1, False, 3000, 520, 520, BF16)),), 255,
                    dtype=torch.uint8, device=DEV)
    for _ in range(3):
        again = M.layernorm_backward(dy, x, gain, out.mean, out.rstd, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        ws.fill_(255)
        assert torch.equal(G, M.weight_grad(dy, out.y_checkpoint, workspace=ws))
        ws.fill_(255)


def test_other_stream():
    x, dy = hidden(600, 256, BF16), grads(600, 256, BF16)
    gain, bias = params(256, BF16)
    want = M.layernorm_forward(x, gain, bias, y_checkpoint="int8")
    want_b = M.layernorm_backward(dy, x, gain, want.mean, want.rstd)
    want_g = M.weight_grad(dy, want.y_checkpoint)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.layernorm_forward(x, gain, bias, y_checkpoint="int8", stream=s)
    got_b = M.layernorm_backward(dy, x, gain, got.mean, got.rstd, stream=s)
    got_g = M.weight_grad(dy, got.y_checkpoint, stream=s)
    back = M.checkpoint_restore(M.checkpoint_save(x, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(want.y, got.y) and torch.equal(want_g, got_g)
    assert all(torch.equal(a, b) for a, b in zip(want_b, got_b))
    assert torch.equal(back, M.checkpoint_restore(M.checkpoint_save(x)))


def test_captured_run():
    """A step's calls captured once and replayed on new inputs."""
    tokens, cols, rows = 512, 256, 384
    gain, bias = params(cols, BF16)
    x, dy, dz = (torch.empty(tokens, n, dtype=BF16, device=DEV) for n in (cols, cols, rows))
    G = torch.zeros(rows, cols, device=DEV)

    def run():
        out = M.layernorm_forward(x, gain, bias, x_checkpoint="e4m3", y_checkpoint="int8")
        M.weight_grad(dz, out.y_checkpoint, G=G, accumulate=True)
        return (out.y, *M.layernorm_backward(dy, out.x_checkpoint, gain, out.mean, out.rstd))

    def fill(seed):
        x.copy_(hidden(tokens, cols, BF16, seed))
        dy.copy_(grads(tokens, cols, BF16, seed))
        dz.copy_(grads(tokens, rows, BF16, seed + 7))

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (1, 2, 3):
        fill(seed)
        G.fill_(seed)
        want = [t.clone() for t in run()]
        want_g = G.clone()
        G.fill_(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)) and torch.equal(want_g, G)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    cases = [weight_case(6000, 520, 264, BF16, "int8", seed=s) for s in (1, 2)]
    off = offsets_of([1000, 0, 5000]).to(DEV)
    want = [M.weight_grad(dy, ck, offsets=off) for dy, ck, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(M.weight_grad(*cases[i][:2], offsets=off, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(want[i], g) for i in (0, 1) for g in got[i])


def test_more_matrices_than_the_plan_sorts():
    counts = [1, 0, 3] * 500
    dy, ck, x64 = weight_case(sum(counts), 24, 40, BF16, "e4m3")
    off = offsets_of(counts)
    check_weight(M.weight_grad(dy, ck, offsets=off.to(DEV)), dy, x64, off.tolist())


def test_copies_of_a_checkpoint():
    x = hidden(70, 200, BF16)
    ck = M.checkpoint_save(x, "int8")
    want = M.checkpoint_restore(ck)
    copies = [copy.copy(ck), copy.deepcopy(ck), pickle.loads(pickle.dumps(ck)),
              M.ActCheckpoint(ck.q.clone(), ck.scale.clone(), 200)]
    copies.append(copy.deepcopy(copies[-1]))
    M.checkpoint_save(torch.zeros_like(x), out=ck)
    assert not M.checkpoint_restore(copies[0]).any()      # a shallow one shares its bytes
    for c in copies[1:]:
        assert c.format == "int8" and c.shape == (70, 200)
        assert torch.equal(M.checkpoint_restore(c), want)


# Rows whose bytes lie past 2^32 elements: the last ones have to be those of a
# short call on the same rows.
FAR, FAR_COLS = 131200, 32768


def test_rows_past_32_bits():
    x = torch.zeros(FAR, FAR_COLS, dtype=BF16, device=DEV)
    x[-40:] = hidden(40, FAR_COLS, BF16)
    gain, bias = params(FAR_COLS, BF16)
    out = M.layernorm_forward(x, gain, bias, x_checkpoint="e4m3", y_checkpoint="int8")
    near = M.layernorm_forward(x[-40:], gain, bias, x_checkpoint="e4m3", y_checkpoint="int8")
    for a, b in zip(out[:3], near[:3]):
        assert torch.equal(a[-40:], b)
    for a, b in zip(out[3:], near[3:]):
        assert torch.equal(a.q[-40:].view(torch.uint8), b.q.view(torch.uint8))
        assert torch.equal(a.scale[-40:], b.scale)
    assert torch.equal(M.checkpoint_restore(out.x_checkpoint)[-40:],
                       M.checkpoint_restore(near.x_checkpoint))
    saved = M.checkpoint_save(x)
    assert torch.equal(saved.q.view(torch.uint8), out.x_checkpoint.q.view(torch.uint8))
    # the other rows' dy is zero, and so is what they add
    dy = torch.zeros_like(x)
    dy[-40:] = grads(40, FAR_COLS, BF16)
    far = M.layernorm_backward(dy, saved, gain, out.mean, out.rstd)
    close = M.layernorm_backward(dy[-40:], near.x_checkpoint, gain, near.mean, near.rstd)
    assert torch.equal(far[0][-40:], close[0]) and not far[0][:-40].any()
    check_backward((close[0], far[1], far[2]), dy[-40:], lo.checkpoint(f64(x[-40:]), "e4m3")[0],
                   gain, near.mean, near.rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols,rows", [(8, FAR_COLS), (8, FAR_COLS - 1), (FAR_COLS, 8)])
def test_weight_grad_past_32_bits(dtype, cols, rows):
    """Whole numbers, so that no order of the sums matters: exact."""
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(FAR, cols, dtype=BF16, device=DEV)
    dy = torch.zeros(FAR, rows, dtype=dtype, device=DEV)
    x[-40:] = torch.randint(-1, 2, (40, cols), generator=g).to(BF16).to(DEV)
    dy[-40:] = torch.randint(-9, 10, (40, rows), generator=g).to(dtype).to(DEV)
    ck = M.checkpoint_save(x, "int8")
    want = dy[-40:].cpu().double().t() @ x[-40:].cpu().double()
    assert torch.equal(M.weight_grad(dy, ck, dtype=F32).cpu().double(), want)
    off = torch.tensor([0, FAR - 50, FAR - 50, FAR], dtype=torch.int64, device=DEV)
    G = M.weight_grad(dy, ck, offsets=off, dtype=F32)
    assert not G[:2].any() and torch.equal(G[2].cpu().double(), want)


@pytest.mark.parametrize("call,error,match", [
    (lambda x, v, ck: M.layernorm_forward(x.t(), v), ValueError, "unit column stride"),
    (lambda x, v, ck: M.layernorm_forward(x, v[:-1]), ValueError, "gain has shape"),
    (lambda x, v, ck: M.layernorm_forward(x, v, v.bfloat16()), TypeError, "bias has dtype"),
    (lambda x, v, ck: M.layernorm_forward(x.half(), v), TypeError, "float32 or bfloat16"),
    (lambda x, v, ck: M.layernorm_forward(x, v, eps=-1.0), M.MuonError, "invalid argument"),
    (lambda x, v, ck: M.layernorm_forward(x, v, x_checkpoint="fp4"), ValueError, "format"),
    (lambda x, v, ck: M.layernorm_forward(x, v, x_checkpoint=ck, y_checkpoint=ck), M.MuonError, "invalid"),
    (lambda x, v, ck: M.layernorm_forward(x[:5], v, x_checkpoint=ck), ValueError, "expected 5 x 64"),
    (lambda x, v, ck: M.layernorm_forward(x[0:1].expand(8, 64), v), ValueError, "row-major"),
    (lambda x, v, ck: M.layernorm_backward(x, x.bfloat16(), v, x[:, 0], x[:, 0]), TypeError, "x has dtype"),
    (lambda x, v, ck: M.layernorm_backward(x, ck, v, x[:, 0], x[:, 0]), ValueError, "contiguous"),
    (lambda x, v, ck: M.layernorm_backward(x, ck, v, v[:8], v[:8], accumulate=True), ValueError, "needs dgain"),
    (lambda x, v, ck: M.layernorm_backward(x, ck, v, v[:8], v[:8], bias=False, dbias=v), ValueError, "bias=False"),
    (lambda x, v, ck: M.weight_grad(x, ck, offsets=torch.zeros(3, dtype=torch.int64, device=DEV), workspace=v[:4]),
     ValueError, "workspace holds"),
    (lambda x, v, ck: M.checkpoint_restore(ck, torch.float16), TypeError, "float32 or bfloat16"),
    (lambda x, v, ck: M.checkpoint_restore(ck, out=x.t()), ValueError, "shape"),
    (lambda x, v, ck: M.weight_grad(x[:7], ck), ValueError, "expected 7 x 64"),
    (lambda x, v, ck: M.weight_grad(x, x), TypeError, "ActCheckpoint"),
    (lambda x, v, ck: M.checkpoint_save([1.0], stream=torch.cuda.Stream()), TypeError, "torch.Tensor"),
    (lambda x, v, ck: M.checkpoint_save(x.cpu(), stream=torch.cuda.Stream()), ValueError, "stream is on"),
    (lambda x, v, ck: M.checkpoint_restore(ck, out=[1.0]), TypeError, "torch.Tensor"),
    (lambda x, v, ck: M.weight_grad(x, ck, accumulate=True), ValueError, "needs G"),
    (lambda x, v, ck: M.weight_grad(x, ck, G=x), ValueError, "G must be"),
    (lambda x, v, ck: M.weight_grad(x, ck, offsets=torch.zeros(3, dtype=torch.int32, device=DEV)), TypeError, "int64"),
    (lambda x, v, ck: M.weight_grad(x, ck, offsets=torch.zeros(3, dtype=torch.int64)), ValueError, "offsets is on"),
])
def test_refusals(call, error, match):
    x, v = hidden(8, 64, F32), torch.ones(64, device=DEV)
    ck = M.checkpoint_save(x)
    with pytest.raises(error, match=match):
        call(x, v, ck)


# -------------------------------------------- a run of them, and the steps
@pytest.mark.parametrize("fmt", FMTS)
def test_layer_to_optimizer_step(fmt):
    """Norm, projection and experts backward into one hybrid optimizer step:
    the steps read the gradients that the operators wrote."""
    tokens, cols, rows, experts = 384, 128, 256, 3
    x = hidden(tokens, cols, BF16, seed=1)
    gain, bias = (torch.nn.Parameter(p) for p in params(cols, BF16))
    W = torch.nn.Parameter(hidden(rows, cols, BF16, seed=2, scale=0.02))
    E = hidden(experts * rows, cols, BF16, seed=3, scale=0.02).view(experts, rows, cols)
    off = torch.tensor([0, 100, 100, tokens], dtype=torch.int64, device=DEV)
    dz, de = grads(tokens, rows, BF16, seed=4), grads(tokens, rows, BF16, seed=5)

    out = M.layernorm_forward(x, gain.data, bias.data, x_checkpoint=fmt, y_checkpoint=fmt)
    W.grad = M.weight_grad(dz, out.y_checkpoint)
    EG = M.weight_grad(de, out.y_checkpoint, offsets=off)
    dy = dz @ W.data
    dx, gain.grad, bias.grad = M.layernorm_backward(dy, out.x_checkpoint, gain.data, out.mean,
                                                    out.rstd)
    y64 = lo.checkpoint(f64(out.y), fmt)[0]
    check_weight(W.grad, dz, y64)
    check_weight(EG, de, y64, off.tolist())
    check_backward((dx, gain.grad, bias.grad), dy, lo.checkpoint(f64(x), fmt)[0], gain.data,
                   out.mean, out.rstd)

    opt = M.HybridMuonAdamW([W], [{"params": [gain, bias], "lr": 0.015}])
    held = [p.detach().clone() for p in (W, gain, bias)]
    E0, EM = E.clone(), torch.zeros(E.shape, device=DEV)
    opt.step()
    M.muon_step_grouped([M.stacked_group(E, EG, EM)], BF16, weight_decay=0.0)
    torch.cuda.synchronize()
    assert all(bool(p.isfinite().all()) and not torch.equal(p, h)
               for p, h in zip((W, gain, bias), held))
    # the expert without a token: zero gradient, zero momentum, no step
    assert torch.equal(E[1], E0[1]) and not torch.equal(E[0], E0[0])
    assert torch.equal(EM[0], EG[0].float()) and not EM[1].any()
