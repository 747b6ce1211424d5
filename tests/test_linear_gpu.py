"""The linear products and weights in 8 bits on the GPU against the fp64 oracle."""
import copy

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from _linear import DEV, check, draw, eight, f64, off, ragged
from oracle import linear_oracle as lin

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# tokens, cols, rows: odd, whole chunks with ends inside a step, whole steps,
# several tiles, the widths of the models
SIZES = [(1, 1, 1), (3, 5, 7), (17, 64, 64), (33, 40, 24), (128, 128, 128), (129, 72, 136),
         (130, 100, 257), (257, 264, 300), (64, 1411, 777), (1, 2048, 1408), (5, 512, 1024)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("tokens,cols,rows", SIZES)
def test_one_matrix(tokens, cols, rows, across, dtype):
    W = draw(rows, cols, dtype=dtype, seed=1)
    x = draw(tokens, rows if across else cols, dtype=dtype, seed=2)
    y = (M.linear_input_grad if across else M.linear_forward)(x, W)
    assert y.dtype == dtype
    check(y, f64(x), f64(W), None, across, dtype, exact_products=dtype == BF16)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("tokens,cols,rows", SIZES)
def test_one_matrix_8_bits(tokens, cols, rows, across, out):
    W = draw(rows, cols, seed=1, scale=0.03)
    x = draw(tokens, rows if across else cols, dtype=F32, seed=2)
    ck, w8, xv, wv = eight(x, W)
    y = (M.linear_input_grad if across else M.linear_forward)(ck, w8, dtype=out)
    assert y.dtype == out
    check(y, xv, wv, None, across, out, eight=True)


RAGGED = [(1, 64, 72, 3, 0, 0), (40, 96, 64, 9, 0, 0), (300, 72, 200, 7, 11, 37),
          (1000, 77, 133, 5, 3, 0), (4000, 136, 264, 3, 0, 100), (2100, 64, 40, 66, 1, 1),
          (3000, 32, 48, 300, 0, 7), (2600, 128, 256, 4, 0, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("tokens,cols,rows,count,before,behind", RAGGED)
def test_ragged(tokens, cols, rows, count, before, behind, across, dtype):
    W = draw(count, rows, cols, dtype=dtype, seed=3)
    x = draw(tokens, rows if across else cols, dtype=dtype, seed=4)
    o = ragged(tokens, count, 5, before, behind)
    y = (M.linear_input_grad if across else M.linear_forward)(x, W, offsets=off(o))
    check(y, f64(x), f64(W), o, across, dtype, exact_products=dtype == BF16)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("tokens,cols,rows,count,before,behind", RAGGED)
def test_ragged_8_bits(tokens, cols, rows, count, before, behind, across, out):
    W = draw(count, rows, cols, seed=3, scale=0.03)
    x = draw(tokens, rows if across else cols, seed=4)
    o = ragged(tokens, count, 5, before, behind)
    ck, w8, xv, wv = eight(x, W)
    y = (M.linear_input_grad if across else M.linear_forward)(ck, w8, offsets=off(o), dtype=out)
    check(y, xv, wv, o, across, out, eight=True)


@pytest.mark.parametrize("offsets", [[-5, 3, 2, 100], [50, 10, 20, 30], [0, 0, 0, 0], [64, 64, 64, 64],
                                     [1 << 62, -(1 << 62), 5, 7], [0, 200, 10, 64]])
@pytest.mark.parametrize("eight_bits", [False, True])
def test_any_offsets_stay_inside(offsets, eight_bits):
    """Offsets outside the tokens or decreasing are read as documented."""
    W, x = draw(3, 40, 72, seed=3), draw(64, 72, seed=4)
    if eight_bits:
        ck, w8, xv, wv = eight(x, W)
        check(M.linear_forward(ck, w8, offsets=off(offsets), dtype=F32), xv, wv, offsets, False, F32, eight=True)
    else:
        check(M.linear_forward(x, W, offsets=off(offsets)), f64(x), f64(W), offsets, False, BF16)
        dy = draw(64, 40, seed=5)
        check(M.linear_input_grad(dy, W, offsets=off(offsets)), f64(dy), f64(W), offsets, True, BF16)


def test_counts_at_the_ends():
    x, W = draw(50, 64, seed=1), draw(1024, 16, 64, seed=2)
    o = np.sort(np.random.default_rng(0).integers(0, 51, 1025)).tolist()
    check(M.linear_forward(x, W, offsets=off(o)), f64(x), f64(W), o, False, BF16)
    with pytest.raises(M.MuonError) as e:
        M.linear_forward(x, draw(1025, 16, 64), offsets=torch.zeros(1026, dtype=torch.int64, device=DEV))
    assert e.value.status == 2
    y = M.linear_forward(x, W[:0], offsets=off([20]))      # no matrix: zeros
    assert y.shape == (50, 16) and not y.any()
    w8 = M.weight_quantize(W[:0])
    assert w8.shape == (0, 16, 64)
    assert not M.linear_forward(M.checkpoint_save(x), w8, offsets=off([7])).any()
    assert M.linear_forward(x[:0], W[0]).shape == (0, 16)
    assert M.linear_input_grad(draw(0, 16), W[:3], offsets=off([0, 0, 0, 0])).shape == (0, 64)
    assert M.linear_forward(M.checkpoint_save(x[:0]), M.weight_quantize(W[0])).shape == (0, 16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("tokens", [20, 200, 1500])
def test_strides_alignment_and_neighbours(dtype, across, tokens):
    """Rows of a wider buffer, starting anywhere, and an output between others:
    the contiguous call's bits, nothing else written or of influence."""
    rows, cols = 136, 264
    k, n = (rows, cols) if across else (cols, rows)
    fn = M.linear_input_grad if across else M.linear_forward
    W, x = draw(rows, cols, dtype=dtype, seed=1), draw(tokens, k, dtype=dtype, seed=2)
    want = fn(x, W)
    check(want, f64(x), f64(W), None, across, dtype, exact_products=dtype == BF16)
    for at, wide in ((0, k + 8), (1, k + 3), (8, k + 24), (5, k + 40)):
        buf = torch.full((tokens, wide), float("nan"), dtype=dtype, device=DEV)
        buf[:, at:at + k] = x
        got = fn(buf[:, at:at + k], W)
        check(got, f64(x), f64(W), None, across, dtype, exact_products=dtype == BF16)
        if at % 8 == 0:
            assert torch.equal(got, want)
    for shift in (0, 1, 3):
        flat = torch.full((tokens * n + 64,), 7.0, dtype=dtype, device=DEV)
        out = flat[32 + shift:32 + shift + tokens * n].view(tokens, n)
        assert fn(x, W, out=out) is out
        assert torch.equal(out, want)
        assert bool((flat[:32 + shift] == 7).all()) and bool((flat[32 + shift + tokens * n:] == 7).all())
    flat = torch.full((rows * cols + 64,), float("nan"), dtype=dtype, device=DEV)
    flat[3:3 + rows * cols] = W.view(-1)
    check(fn(x, flat[3:3 + rows * cols].view(rows, cols)), f64(x), f64(W), None, across, dtype,
          exact_products=dtype == BF16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens,k", [(30, 72), (300, 72), (300, 77), (1500, 72)])
@pytest.mark.parametrize("across", [False, True])
def test_bad_values_stay_in_their_rows(bad, tokens, k, across):
    """A NaN or infinity in a token reaches that token's outputs only; in a
    weight, the outputs of its row (column) for that matrix's tokens only.  What
    a padded step or a neighbouring matrix holds reaches nothing."""
    n = 96
    fn = M.linear_input_grad if across else M.linear_forward
    W = draw(3, *((k, n) if across else (n, k)), seed=1)
    x = draw(tokens, k, seed=2)
    o = [4, tokens // 2, tokens // 2, tokens - 3]
    clean = fn(x, W, offsets=off(o))
    xb = x.clone()
    xb[0] = bad                       # of no matrix
    xb[tokens // 2 - 1, k - 1] = bad
    xb[tokens - 1] = bad              # of no matrix
    Wb = W.clone()
    Wb[1] = bad                       # no token takes it
    y = fn(xb, Wb, offsets=off(o))
    hit = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    hit[tokens // 2 - 1] = True
    assert torch.equal(y[~hit], clean[~hit])
    want = f64(x)[tokens // 2 - 1] * 0
    with np.errstate(invalid="ignore"):
        xr = f64(xb)[tokens // 2 - 1]
        want = xr @ (f64(W)[0] if across else f64(W)[0].T)
    got = f64(y)[tokens // 2 - 1]
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    Wb = W.clone()
    Wb[(0, k - 1, 5) if across else (0, 5, k - 1)] = bad
    y = fn(x, Wb, offsets=off(o))
    fine = torch.ones_like(clean, dtype=torch.bool)
    fine[4:tokens // 2, 5] = False
    assert torch.equal(y[fine], clean[fine])
    assert not bool(torch.isfinite(y[4:tokens // 2, 5]).any())


@pytest.mark.parametrize("out", [BF16, F32])
def test_marked_blocks_of_8_bits(out):
    """A checkpoint's marked block makes its token NaN, a weight's marked block
    the outputs that it reaches; nothing else."""
    x, W = draw(200, 300, seed=1), draw(300, 300, seed=2)
    clean = M.linear_forward(M.checkpoint_save(x), M.weight_quantize(W), dtype=out)
    xb, Wb = x.clone(), W.clone()
    xb[17, 299] = float("nan")
    Wb[140, 10] = float("inf")
    y = M.linear_forward(M.checkpoint_save(xb), M.weight_quantize(Wb), dtype=out)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[17] = True
    hit[:, 128:256] = True
    assert torch.equal(torch.isnan(y), hit) and torch.equal(y[~hit], clean[~hit])
    dx = M.linear_input_grad(M.checkpoint_save(x), M.weight_quantize(Wb), dtype=out)
    assert bool(torch.isnan(dx[:, :128]).all()) and not bool(torch.isnan(dx[:, 128:]).any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1), (7, 5), (128, 128), (129, 127), (300, 77), (2, 200, 264), (3, 1, 400)])
def test_weights_in_8_bits(shape, dtype):
    """Every byte of q, q_t and scale, paddings included."""
    W = draw(*shape, dtype=dtype, seed=7, scale=0.02)
    W.view(-1)[0] = 0.875 * 2.0 ** -3       # a power of two times the largest number
    w8 = M.weight_quantize(W)
    assert w8.shape == tuple(shape)
    stack = f64(W).reshape((-1,) + tuple(shape[-2:]))
    q = f64(w8.q).reshape((-1,) + tuple(w8.q.shape[-2:]))
    q_t = f64(w8.q_t).reshape((-1,) + tuple(w8.q_t.shape[-2:]))
    scale = w8.scale.cpu().numpy().reshape((-1,) + tuple(w8.scale.shape[-2:]))
    rows, cols = shape[-2:]
    for e, w in enumerate(stack):
        _, want, s = lin.quantized(w)
        assert np.array_equal(scale[e], s)
        assert np.array_equal(q[e, :, :cols], want) and not q[e, :, cols:].any()
        assert np.array_equal(q_t[e, :, :rows], want.T) and not q_t[e, :, rows:].any()
    again = M.weight_quantize(W, out=M.Weight8.empty(*shape, device=DEV))
    assert torch.equal(again.q_t.view(torch.uint8), w8.q_t.view(torch.uint8))


def test_weights_in_8_bits_at_the_ends_of_float32():
    W = torch.zeros(128 * 5, 128, device=DEV)
    W[0, 0], W[128, 1], W[256, 2], W[384, 3] = 3.4e38, 2.0 ** -149, 448 * 2.0 ** -117, float("-inf")
    W[384, 4] = 1.0
    w8 = M.weight_quantize(W)
    _, q, scale = lin.quantized(f64(W))
    assert np.array_equal(w8.scale.cpu().numpy(), scale) and scale[:, 0].tolist() == [246, 10, 10, 255, 10]
    assert np.array_equal(f64(w8.q), q) and np.array_equal(f64(w8.q_t), q.T)


def test_large_and_small_scales_in_a_product():
    """Scales far apart, in k and between operands: they meet in float32."""
    for out in (F32, BF16):
        x, W = draw(70, 256, dtype=F32, seed=1), draw(140, 256, dtype=F32, seed=2)
        x = x * torch.exp2(torch.linspace(-60, 60, 8, device=DEV)).repeat_interleave(32)
        W = W * torch.exp2(torch.tensor([40.0, -40.0], device=DEV)).repeat_interleave(128)
        ck, w8, xv, wv = eight(x, W)
        check(M.linear_forward(ck, w8, dtype=out), xv, wv, None, False, out, eight=True)


def test_rows_past_32_bits():
    """Inputs and outputs of more than 2^32 bytes and 2^31 elements."""
    tokens, k, n = 70_000, 32768, 72
    x = torch.zeros(tokens, k, dtype=BF16, device=DEV)
    pick = [0, 1, 4097, 65535, 65536, 69_998, 69_999]
    rows = draw(len(pick), k, seed=1)
    x[pick] = rows
    W = draw(n, k, seed=2)
    y = M.linear_forward(x, W)
    check(y[pick], f64(rows), f64(W), None, False, BF16)
    rest = torch.ones(tokens, dtype=torch.bool, device=DEV)
    rest[pick] = False
    assert not bool(y[rest].any())
    ck = M.checkpoint_save(x)
    del x
    xv = f64(M.checkpoint_restore(M.checkpoint_save(rows), F32))
    w8 = M.weight_quantize(W)
    check(M.linear_forward(ck, w8)[pick], xv, lin.quantized(f64(W))[0], None, False, BF16, eight=True)
    del ck
    dy = torch.zeros(tokens, n, dtype=BF16, device=DEV)
    small = draw(len(pick), n, seed=3)
    dy[pick] = small
    dx = M.linear_input_grad(dy, W)
    check(dx[pick], f64(small), f64(W), None, True, BF16)
    assert not bool(dx[40_000].any())


def test_a_row_stride_past_32_bits():
    """A stride of 2^23 elements and more: bytes within a tile leave 32 bits."""
    for ld in (1 << 23, 1 << 24):
        buf = torch.empty(300 * ld, dtype=BF16, device=DEV)
        x = buf.as_strided((300, 64), (ld, 1))
        v = draw(300, 64, seed=1)
        x.copy_(v)
        W = draw(80, 64, seed=2)
        check(M.linear_forward(x, W), f64(v), f64(W), None, False, BF16)
        del buf, x


@pytest.mark.parametrize("eight_bits", [False, True])
def test_deterministic_and_independent_of_neighbours(eight_bits):
    """The same bits on every run."""
    x, W = draw(1500, 200, seed=1), draw(6, 136, 200, seed=2)
    o = off(ragged(1500, 6, 3))
    a, w = (M.checkpoint_save(x), M.weight_quantize(W)) if eight_bits else (x, W)
    first = M.linear_forward(a, w, offsets=o)
    for _ in range(3):
        assert torch.equal(M.linear_forward(a, w, offsets=o), first)


@pytest.mark.parametrize("tokens", [6, 300])
def test_streams_and_graphs(tokens):
    """On another stream; captured, and replayed with other values, offsets among
    them, between eager work."""
    x, W = draw(tokens, 72, seed=1), draw(4, 136, 72, seed=2)
    dy = draw(tokens, 136, seed=3)
    o = off(ragged(tokens, 4, 5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = M.linear_forward(x, W, offsets=o, stream=side)
    side.synchronize()
    assert torch.equal(y, M.linear_forward(x, W, offsets=o))
    graph = torch.cuda.CUDAGraph()
    w8 = M.Weight8.empty(4, 136, 72, device=DEV)
    with torch.cuda.graph(graph):
        y = M.linear_forward(x, W, offsets=o)
        dx = M.linear_input_grad(dy, W, offsets=o)
        M.weight_quantize(W, out=w8)
        y8 = M.linear_forward(M.checkpoint_save(x), w8, offsets=o)
        dx8 = M.linear_input_grad(M.checkpoint_save(dy), w8, offsets=o)
    for k in range(3):
        x.copy_(draw(tokens, 72, seed=10 + k))
        W.copy_(draw(4, 136, 72, seed=20 + k))
        o.copy_(off(ragged(tokens, 4, 30 + k)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, M.linear_forward(x, W, offsets=o))
        assert torch.equal(dx, M.linear_input_grad(dy, W, offsets=o))
        w = M.weight_quantize(W)
        assert torch.equal(y8, M.linear_forward(M.checkpoint_save(x), w, offsets=o))
        assert torch.equal(dx8, M.linear_input_grad(M.checkpoint_save(dy), w, offsets=o))


def test_copies_of_weights_in_8_bits():
    w8 = M.weight_quantize(draw(130, 70))
    other = copy.deepcopy(w8)
    assert other.shape == w8.shape and other.q.data_ptr() != w8.q.data_ptr()
    x = M.checkpoint_save(draw(5, 70))
    assert torch.equal(M.linear_forward(x, other), M.linear_forward(x, w8))
    assert w8.nbytes == 130 * 128 + 70 * 256 + 2


def test_front_end_refusals():
    x, W = draw(20, 64), draw(40, 64)
    ck, w8 = M.checkpoint_save(x), M.weight_quantize(W)
    o = off([0, 10, 20])
    stack = draw(2, 40, 64)
    for call, error in [
        (lambda: M.linear_forward(x, w8), TypeError), (lambda: M.linear_forward(ck, W), TypeError),
        (lambda: M.linear_forward(x, W.float()), TypeError),
        (lambda: M.linear_forward(x, W, dtype=torch.float32), TypeError),
        (lambda: M.linear_forward(ck, w8, dtype=torch.float16), TypeError),
        (lambda: M.linear_forward(x.half(), W.half()), TypeError),
        (lambda: M.linear_forward(M.checkpoint_save(x, "int8"), w8), ValueError),
        (lambda: M.linear_forward(x[:, :60], W), ValueError),
        (lambda: M.linear_input_grad(x, W), ValueError),
        (lambda: M.linear_forward(x, W.t().contiguous().t()), ValueError),
        (lambda: M.linear_forward(x.t(), draw(4, 20)), ValueError),
        (lambda: M.linear_forward(x, W, offsets=o), ValueError),
        (lambda: M.linear_forward(x, stack), ValueError),
        (lambda: M.linear_forward(x, stack, offsets=o[:2]), ValueError),
        (lambda: M.linear_forward(x, stack, offsets=o.int()), TypeError),
        (lambda: M.linear_forward(x, stack, offsets=o.cpu()), ValueError),
        (lambda: M.linear_forward(x, W, out=draw(20, 41)), ValueError),
        (lambda: M.linear_forward(x, W, out=draw(20, 40, dtype=torch.float32)), TypeError),
        (lambda: M.linear_forward(x, W.cpu()), ValueError),
        (lambda: M.weight_quantize(W.t()), ValueError), (lambda: M.weight_quantize(W[0]), ValueError),
        (lambda: M.weight_quantize(W.half()), TypeError),
        (lambda: M.weight_quantize(W, out=M.Weight8.empty(40, 65, device=DEV)), ValueError),
        (lambda: M.Weight8(w8.q, w8.q_t[:, :64], w8.scale), ValueError),
        (lambda: M.Weight8(w8.q.view(torch.uint8), w8.q_t, w8.scale), TypeError),
        (lambda: M.Weight8.empty(0, 5), ValueError), (lambda: M.Weight8.empty(4), ValueError),
    ]:
        with pytest.raises(error):
            call()
    with pytest.raises(M.MuonError):      # an output over its input
        M.linear_forward(x, draw(64, 64), out=x)


def test_outputs_that_autograd_kept_are_noticed():
    x, W = draw(20, 64), draw(64, 64)
    y = torch.ones(20, 64, dtype=BF16, device=DEV, requires_grad=True)
    z = y * 2
    keep = (z * z).sum()
    M.linear_forward(x, W, out=z.detach())
    with pytest.raises(RuntimeError, match="modified"):
        keep.backward()


@pytest.mark.parametrize("tokens", [3, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_subnormal_operands(dtype, tokens):
    """x of 1 .. 63 steps of 2^-133 (bf16's smallest number), W a power of two: sums of
    one product each are exact."""
    g = torch.Generator().manual_seed(2)
    x = torch.zeros(tokens, 96)
    at = torch.randint(0, 96, (tokens,), generator=g)
    x[torch.arange(tokens), at] = torch.randint(1, 64, (tokens,), generator=g).float() * 2.0 ** -133
    x = x.to(dtype).to(DEV)
    W = torch.full((80, 96), 2.0 ** 20, dtype=dtype, device=DEV)
    want = (f64(x).sum(1) * 2.0 ** 20)[:, None] * np.ones(80)
    assert (want > 0).all()
    assert np.array_equal(f64(M.linear_forward(x, W)), want)
    V = torch.full((96, 80), 2.0 ** 20, dtype=dtype, device=DEV)
    assert np.array_equal(f64(M.linear_input_grad(x, V)), want)
