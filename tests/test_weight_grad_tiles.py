"""The 256 x 256 tiles of the weight gradient.

Which tiles a call takes is the choice of an estimate, so each test asserts that
its sizes still take the large ones: on the CPU, and again where it runs.
"""
import os

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib

from test_layer_extremes_gpu import SIZES as EXTREMES
from _layers import DEV, check_weight, f64, grads, hidden

BF16, F32 = torch.bfloat16, torch.float32
FMTS = ["e4m3", "int8"]


def tile(count, tokens, rows, cols, dtype=BF16, ragged=True):
    return _lib.lib().muon_weight_grad_tile(count, int(ragged), tokens, rows, cols,
                                            M.api.dtype_code(dtype))


# Steps of 32 tokens: from one to eleven, whole and not, by themselves ...
STEPS = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 161, 192, 200, 224, 255, 256,
         257, 288, 300, 320, 352]
STEPS_ROWS, STEPS_COLS = 4096, 4096
# ... and as the matrices of one call, which cuts the longer ones; columns and
# rows that end inside a tile
COUNTS = [0, 1, 31, 32, 33, 64, 65, 95, 96, 97, 127, 128, 129, 160, 191, 192, 224, 255, 256, 288,
          320, 352, 353, 0]
COUNTS_SIZES = [(1032, 520), (2056, 1032)]
# whole tiles, rows and columns that end inside one, and rows repacked first
APART = [(2048, 1024), (2040, 1020), (2051, 2050)]
MANY = [(100, 5000, 1024, 512), (100, 5000, 1016, 520), (1100, 22000, 256, 256),
        (1100, 22000, 251, 256)]
FAR = 131200      # times 32768 columns: past 2^32
FAR_SIZES = [(32768, 256), (32760, 264), (256, 32768), (264, 32760)]
TWICE = (9000, 2048, 1024)


@pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmuon.so not built")
def test_the_sizes_here_take_the_large_tiles():
    for t in STEPS:
        assert tile(1, t, STEPS_ROWS, STEPS_COLS, ragged=False) == 256, t
    for rows, cols in COUNTS_SIZES:
        assert tile(len(COUNTS), sum(COUNTS) + 7, rows, cols) == 256, (rows, cols)
    for rows, cols in APART:
        assert tile(3, 9000, rows, cols) == 256, (rows, cols)
    for count, tokens, rows, cols in MANY:
        assert tile(count, tokens, rows, cols) == 256, (count, rows, cols)
    for rows, cols in FAR_SIZES:
        assert tile(1, FAR, rows, cols, ragged=False) == tile(3, FAR, rows, cols) == 256, (rows, cols)
    assert tile(3, *TWICE) == 256
    assert tile(1, *EXTREMES[1], ragged=False) == 256
    # float32 dy takes the small ones, and so do small matrices
    assert tile(1, 16384, 4096, 1024, F32, False) == 128 == tile(1, 96, 768, 768, BF16, False)
    # sizes that are refused
    for bad in ((0, 5, 5, 5), (1, -1, 5, 5), (1, 5, 0, 5), (1, 5, 5, _lib.MUON_MAX_DIM + 1)):
        assert tile(*bad) == 0
    assert _lib.lib().muon_weight_grad_tile(1, 0, 5, 5, 5, 7) == 0


def integers(tokens, rows, cols, seed):
    """Whole numbers whose sums stay under 2^24: float32 sums of them are exact
    in any order."""
    g = torch.Generator().manual_seed(seed)
    dy = torch.randint(-64, 65, (tokens, rows), generator=g).to(BF16).to(DEV)
    x = torch.randint(-3, 4, (tokens, cols), generator=g).to(BF16).to(DEV)
    return dy, x


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_every_number_of_steps(fmt):
    for t in STEPS:
        dy, x = integers(t, STEPS_ROWS, STEPS_COLS, t)
        assert tile(1, t, STEPS_ROWS, STEPS_COLS, ragged=False) == 256
        got = M.weight_grad(dy, M.checkpoint_save(x, fmt), dtype=F32)
        assert torch.equal(got.double(), dy.t().double() @ x.double()), t


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", COUNTS_SIZES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gdtype", [BF16, F32])
def test_every_number_of_steps_at_once(rows, cols, fmt, gdtype):
    tokens = sum(COUNTS) + 7      # tokens that belong to nobody
    dy, x = integers(tokens, rows, cols, rows)
    off = [0] + np.cumsum(COUNTS).tolist()
    assert tile(len(COUNTS), tokens, rows, cols) == 256
    before = torch.randint(-9, 10, (len(COUNTS), rows, cols), device=DEV).to(gdtype)
    into = before.clone()
    at = torch.tensor(off, dtype=torch.int64, device=DEV)
    ck = M.checkpoint_save(x, fmt)
    G = M.weight_grad(dy, ck, offsets=at, dtype=gdtype)
    M.weight_grad(dy, ck, offsets=at, G=into, accumulate=True)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        want = dy[a:b].t().double() @ x[a:b].double()
        assert torch.equal(G[e], want.to(gdtype)), e
        assert torch.equal(into[e], (want + before[e].double()).to(gdtype)), e


@pytest.mark.gpu
@pytest.mark.parametrize("start,more", [(8, 16), (3, 16), (8, 17)])
def test_rows_that_the_large_tiles_cannot_read(start, more):
    """A ragged call whose sizes take the large tiles, dy a view whose rows start
    on 16 bytes, start elsewhere, or are an odd stride apart: the same bits."""
    rows, cols = COUNTS_SIZES[0]
    tokens = sum(COUNTS) + 7
    assert tile(len(COUNTS), tokens, rows, cols) == 256
    dy, x = integers(tokens, rows, cols, 5)
    ck = M.checkpoint_save(x, "int8")
    at = torch.tensor([0] + np.cumsum(COUNTS).tolist(), dtype=torch.int64, device=DEV)
    wide = torch.full((tokens, rows + more), float("nan"), dtype=BF16, device=DEV)
    view = wide[:, start:start + rows]
    view.copy_(dy)
    want = M.weight_grad(dy, ck, offsets=at, dtype=F32)
    assert torch.equal(M.weight_grad(view, ck, offsets=at, dtype=F32), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", APART)
def test_bad_tokens_stay_apart(rows, cols):
    """Marked blocks, NaN and infinities of one matrix's tokens, and of its
    neighbours' in the same steps."""
    tokens = 9000
    assert tile(3, tokens, rows, cols) == 256
    dy, x = grads(tokens, rows, BF16, seed=6), hidden(tokens, cols, BF16, seed=6)
    off = torch.tensor([0, 3001, 3002, 9000], dtype=torch.int64, device=DEV)
    clean = M.weight_grad(dy, M.checkpoint_save(x, "int8"), offsets=off)
    dy[3001, :] = float("nan")
    x[3001, 40] = float("inf")
    for fmt in FMTS:
        got = M.weight_grad(dy, M.checkpoint_save(x, fmt), offsets=off)
        assert bool(got[1].isnan().all()) and not bool(got[[0, 2]].isnan().any())
        if fmt == "int8":
            assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    dy[3001, :] = 1.0
    dy[3001, 5] = float("inf")
    x[3001, 40] = 2.0
    x[3001, 64:96] = float("inf")      # a marked block
    x[3001, 96:128] = 3.0
    x[3001, cols - 1] = float("nan")   # one that the row's end cuts
    last = (cols - 1) // 32 * 32
    for fmt in FMTS:
        got = M.weight_grad(dy, M.checkpoint_save(x, fmt), offsets=off)
        assert bool(got[1][:, 64:96].isnan().all()) and not bool(got[[0, 2]].isnan().any())
        assert bool(got[1][:, last:].isnan().all())
        assert bool((got[1][5, 96:128] == float("inf")).all())
        others = torch.arange(rows) != 5
        assert bool((got[1][others][:, 96:128] == 3.0).all())
    # in the first and the last token of a longer matrix: its own columns only
    dy[3001, 5] = 1.0
    x[3001] = 1.0
    for token in (3002, 8999):
        bad = x.clone()
        bad[token, 128:160] = float("nan")
        got = M.weight_grad(dy, M.checkpoint_save(bad, "int8"), offsets=off)
        assert bool(got[2][:, 128:160].isnan().all()) and not bool(got[:2].isnan().any())
        assert torch.equal(got[2][:, :128], clean[2][:, :128])
        assert torch.equal(got[2][:, 160:], clean[2][:, 160:])


@pytest.mark.gpu
@pytest.mark.parametrize("count,tokens,rows,cols", MANY)
def test_more_matrices_than_a_wave_plans(count, tokens, rows, cols):
    """More than 64, and (1100) more than the plan puts in order: uneven ones,
    some without a token."""
    g = torch.Generator().manual_seed(count)
    share = torch.rand(count, generator=g) ** 3 * (torch.rand(count, generator=g) < 0.9)
    counts = torch.bincount(torch.multinomial(share, tokens - 5, replacement=True, generator=g),
                            minlength=count)
    off = [0] + counts.cumsum(0).tolist()
    assert tile(count, tokens, rows, cols) == 256
    dy, x = integers(tokens, rows, cols, count)
    G = M.weight_grad(dy, M.checkpoint_save(x, "e4m3"), dtype=F32,
                      offsets=torch.tensor(off, dtype=torch.int64, device=DEV))
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        assert torch.equal(G[e].double(), dy[a:b].t().double() @ x[a:b].double()), e


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", FAR_SIZES)
def test_rows_past_32_bits(rows, cols):
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(FAR, cols, dtype=BF16, device=DEV)
    dy = torch.zeros(FAR, rows, dtype=BF16, device=DEV)
    x[-40:] = torch.randint(-1, 2, (40, cols), generator=g).to(BF16).to(DEV)
    dy[-40:] = torch.randint(-9, 10, (40, rows), generator=g).to(BF16).to(DEV)
    ck = M.checkpoint_save(x, "int8")
    want = dy[-40:].t().double() @ x[-40:].double()
    assert tile(1, FAR, rows, cols, ragged=False) == tile(3, FAR, rows, cols) == 256
    assert torch.equal(M.weight_grad(dy, ck, dtype=F32).double(), want)
    off = torch.tensor([0, FAR - 50, FAR - 50, FAR], dtype=torch.int64, device=DEV)
    G = M.weight_grad(dy, ck, offsets=off, dtype=F32)
    assert not G[:2].any() and torch.equal(G[2].double(), want)


@pytest.mark.gpu
def test_two_streams_and_a_replayed_graph():
    tokens, rows, cols = TWICE
    assert tile(3, tokens, rows, cols) == 256
    off = torch.tensor([0, 1000, 1000, 9000], dtype=torch.int64, device=DEV)
    cases = []
    for seed in (1, 2):
        dy = grads(tokens, rows, BF16, seed)
        cases.append((dy, M.checkpoint_save(hidden(tokens, cols, BF16, seed), "int8")))
    want = [M.weight_grad(dy, ck, offsets=off) for dy, ck in cases]
    for (dy, ck), G in zip(cases, want):
        check_weight(G, dy, f64(M.checkpoint_restore(ck, F32)), off.tolist())
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(M.weight_grad(*cases[i], offsets=off, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(want[i], g) for i in (0, 1) for g in got[i])
    # captured on one input and its offsets, replayed on others
    dy, ck = cases[0][0].clone(), copy_of(cases[0][1])
    at = off.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = M.weight_grad(dy, ck, offsets=at)
    for i, moved in ((1, [0, 9000, 9000, 9000]), (0, [5, 40, 3000, 9000]), (1, [0, 1000, 1000, 9000])):
        dy.copy_(cases[i][0])
        ck.q.copy_(cases[i][1].q)
        ck.scale.copy_(cases[i][1].scale)
        at.copy_(torch.tensor(moved, dtype=torch.int64))
        eager = M.weight_grad(*cases[i], offsets=at)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, eager)


def copy_of(ck):
    return M.ActCheckpoint(ck.q.clone(), ck.scale.clone(), ck.cols)


@pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmuon.so not built")
@pytest.mark.parametrize("tokens,rows,cols", [(65536, 1001, 8), (65536, 1000, 8), (16384, 4096, 1024),
                                              (16384, 4095, 1024), (2049, 1001, 777), (96, 768, 768)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_workspace_holds_partial_sums_and_repacked_rows(tokens, rows, cols, dtype):
    """At most 64 parts of one matrix, each G in float32; dy once more, in padded
    rows of bf16, only where the large tiles take odd ones.  (float32 dy is split
    on its way to LDS and needs no room.)"""
    got = M.weight_grad_workspace_bytes(1, False, tokens, rows, cols, dtype)
    repacked = dtype == BF16 and rows % 8 != 0 and tile(1, tokens, rows, cols, dtype, False) == 256
    room = tokens * (rows + 7) // 8 * 8 * 2 if repacked else 0
    assert room * 0.99 <= got <= 64 * rows * cols * 4 + room + 1024
