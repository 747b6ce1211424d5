"""Calls of the layer operators that the interface allows at its edges: odd
addresses, parts of a checkpoint, no tokens, results past 2^32 elements, the most
matrices, many short rows, graphs that share inputs."""
import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from oracle import layer_oracle as lo

from _layers import (DEV, check_backward, check_forward, check_weight, f64, grads, hidden, params)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FMTS = ["e4m3", "int8"]


def odd(shape, dtype, by=1):
    """A contiguous tensor `by` elements off its allocation's alignment, between
    guards."""
    n = int(np.prod(shape))
    flat = torch.full((n + by + 9,), 7.0, dtype=dtype, device=DEV)
    return flat, flat[by:by + n].view(shape)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(300, 96, 72), (300, 97, 71), (5003, 2056, 1030)])
def test_results_at_odd_addresses(dtype, tokens, rows, cols):
    """Gradients inside a flat buffer, and a workspace that starts anywhere."""
    dy = grads(tokens, rows, dtype, 3)
    ck = M.checkpoint_save(hidden(tokens, cols, dtype, 3), "int8")
    ws = torch.empty(M.weight_grad_workspace_bytes(1, False, tokens, rows, cols, dtype) + 3,
                     dtype=torch.uint8, device=DEV)[3:]
    for gdtype in (BF16, F32):
        want = M.weight_grad(dy, ck, dtype=gdtype)
        for by in (1, 3):
            flat, G = odd((rows, cols), gdtype, by)
            M.weight_grad(dy, ck, G=G, workspace=ws)
            assert torch.equal(G, want)
            assert (flat[:by] == 7).all() and (flat[by + G.numel():] == 7).all()
    gain, bias = params(cols, dtype)
    at, shift = odd((cols,), dtype)[1], odd((cols,), dtype, 3)[1]
    at.copy_(gain), shift.copy_(bias)
    x, d = hidden(tokens, cols, dtype, 4), grads(tokens, cols, dtype, 4)
    out, want = M.layernorm_forward(x, at, shift), M.layernorm_forward(x, gain, bias)
    assert all(torch.equal(a, b) for a, b in zip(out[:3], want[:3]))
    (gf, dgain), (bf, dbias) = odd((cols,), dtype, 5), odd((cols,), dtype)
    ws = torch.empty(M.layernorm_workspace_bytes(tokens, cols) + 1, dtype=torch.uint8, device=DEV)[1:]
    got = M.layernorm_backward(d, x, at, out.mean, out.rstd, dgain=dgain, dbias=dbias, workspace=ws)
    for a, b in zip(got, M.layernorm_backward(d, x, gain, out.mean, out.rstd)):
        assert torch.equal(a, b)
    for flat, by in ((gf, 5), (bf, 1)):
        assert (flat[:by] == 7).all() and (flat[by + cols:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_tokens_of_a_checkpoint(fmt):
    """A checkpoint of some tokens of another, which it shares the bytes with."""
    x, dy = hidden(400, 200, BF16), grads(400, 96, BF16)
    ck = M.checkpoint_save(x, fmt)
    part = M.ActCheckpoint(ck.q[101:357], ck.scale[101:357], 200)
    assert torch.equal(M.checkpoint_restore(part), M.checkpoint_restore(ck)[101:357])
    x64 = f64(M.checkpoint_restore(part, F32))
    check_weight(M.weight_grad(dy[101:357], part), dy[101:357], x64)
    gain, bias = params(200, BF16)
    out = M.layernorm_forward(x[101:357], gain, bias)
    d = grads(256, 200, BF16, seed=4)
    check_backward(M.layernorm_backward(d, part, gain, out.mean, out.rstd), d, x64, gain, out.mean,
                   out.rstd)
    # written in place: the tokens around it stay
    before = ck.q.view(torch.uint8).clone()
    M.checkpoint_save(2 * x[101:357], out=part)
    after = ck.q.view(torch.uint8)
    assert torch.equal(after[:101], before[:101]) and torch.equal(after[357:], before[357:])
    assert torch.equal(M.checkpoint_restore(ck)[101:357], M.checkpoint_restore(part))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_grad_without_a_token(dtype):
    dy = torch.empty(0, 40, dtype=dtype, device=DEV)
    ck = M.checkpoint_save(torch.empty(0, 72, dtype=dtype, device=DEV), "int8")
    assert not M.weight_grad(dy, ck).any()
    off = torch.tensor([0, 0, 5, -3], dtype=torch.int64, device=DEV)
    G = torch.full((3, 40, 72), 3.0, dtype=dtype, device=DEV)
    M.weight_grad(dy, ck, offsets=off, G=G, accumulate=True)
    assert (G == 3).all()
    assert not M.weight_grad(dy, ck, offsets=off, G=G).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_past_32_bits(dtype):
    """A stack of more than 2^32 elements, whole numbers: exact."""
    count, rows, cols, tokens = 5, 32768, 32768, 40
    g = torch.Generator().manual_seed(1)
    dy = torch.randint(-9, 10, (tokens, rows), generator=g).to(dtype).to(DEV)
    x = torch.randint(-3, 4, (tokens, cols), generator=g).to(BF16).to(DEV)
    off = [0, 0, 11, 12, 12, 40]
    G = M.weight_grad(dy, M.checkpoint_save(x, "e4m3"), dtype=BF16,
                      offsets=torch.tensor(off, dtype=torch.int64, device=DEV))
    assert G.numel() > 2 ** 32
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        want = dy[a:b].t().float() @ x[a:b].float()      # under 2^24: exact
        assert torch.equal(G[e], want.to(BF16)), e


def test_most_matrices():
    """2^20 of them, most of one token."""
    count = 1 << 20
    tokens = count - 7
    g = torch.Generator().manual_seed(2)
    dy = torch.randint(-9, 10, (tokens, 3), generator=g).to(BF16).to(DEV)
    x = torch.randint(-9, 10, (tokens, 5), generator=g).to(BF16).to(DEV)
    ends = torch.arange(1, count + 1).clamp(max=tokens)
    ends[1000:1500] = 1500      # one of 501 tokens, 499 of none
    off = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(DEV)
    G = M.weight_grad(dy, M.checkpoint_save(x, "int8"), offsets=off, dtype=F32)
    want = dy.float()[:, :, None] * x.float()[:, None, :]
    assert torch.equal(G[:1000], want[:1000]) and torch.equal(G[1500:tokens], want[1500:])
    assert torch.equal(G[1000], want[1000:1500].sum(0))
    assert not G[1001:1500].any() and not G[tokens:].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [3, 20])
def test_many_short_rows(dtype, cols):
    """More rows than any grid has places; the gradients against 64 bits."""
    tokens = 1_500_001
    x = hidden(1501, cols, dtype, 1).repeat(1000, 1)[:tokens]
    dy = grads(1499, cols, dtype, 1).repeat(1001, 1)[:tokens]
    x, dy = torch.cat([x, x[:tokens - len(x)]]), torch.cat([dy, dy[:tokens - len(dy)]])
    gain, bias = params(cols, F32)
    out = M.layernorm_forward(x, gain, bias, x_checkpoint="int8")
    check_forward(out, x, gain, bias, 1e-5)
    check_backward(M.layernorm_backward(dy, x, gain, out.mean, out.rstd), dy, f64(x), gain, out.mean,
                   out.rstd)
    kept = lo.checkpoint(f64(x), "int8")[0]
    assert np.array_equal(f64(M.checkpoint_restore(out.x_checkpoint, F32)), kept)
    check_backward(M.layernorm_backward(dy, out.x_checkpoint, gain, out.mean, out.rstd), dy, kept,
                   gain, out.mean, out.rstd)


def test_two_graphs_of_one_step():
    """Two graphs captured of the same inputs, replayed in turn and with eager
    calls between them: neither disturbs the other's results."""
    x, dy = hidden(3000, 520, BF16), grads(3000, 520, BF16)
    gain, bias = params(520, F32)

    def run():
        out = M.layernorm_forward(x, gain, bias, x_checkpoint="int8", y_checkpoint="e4m3")
        return (out.y, *M.layernorm_backward(dy, out.x_checkpoint, gain, out.mean, out.rstd),
                M.weight_grad(dy, out.y_checkpoint))

    run()
    torch.cuda.synchronize()
    graphs, held = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(run())
    for seed in (1, 2, 3):
        x.copy_(hidden(3000, 520, BF16, seed))
        first = [t.clone() for t in run()]
        graphs[0].replay()
        dy.copy_(grads(3000, 520, BF16, seed))
        second = [t.clone() for t in run()]
        graphs[1].replay()
        third = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held[0]))
        assert all(torch.equal(a, b) for a, b in zip(second, held[1]))
        assert all(torch.equal(a, b) for a, b in zip(second, third))


def test_one_tensor_for_several_inputs():
    """Inputs may overlap each other: dy = x, one vector as gain and bias."""
    x = hidden(70, 200, BF16)
    v = params(200, BF16)[0]
    out = M.layernorm_forward(x, v, v)
    check_forward(out, x, v, v, 1e-5)
    check_backward(M.layernorm_backward(x, x, v, out.mean, out.rstd), x, f64(x), v, out.mean, out.rstd)
    ck = M.checkpoint_save(x)
    check_weight(M.weight_grad(x, ck), x, f64(M.checkpoint_restore(ck, F32)))


@pytest.mark.parametrize("cols,limit", [(4096, 16), (8192, 3), (16384, 2), (32768, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_on_both_sides_of_one_block(cols, limit, dtype):
    """The last number of rows that a single block takes, and one more."""
    gain, bias = params(cols, dtype)
    for tokens in (limit, limit + 1, limit + 5):
        assert (M.layernorm_workspace_bytes(tokens, cols) == 0) == (tokens == limit)
        x, dy = hidden(tokens, cols, dtype, 1), grads(tokens, cols, dtype, 1)
        out = M.layernorm_forward(x, gain, bias)
        check_backward(M.layernorm_backward(dy, x, gain, out.mean, out.rstd), dy, f64(x), gain,
                       out.mean, out.rstd)
        dgain, dbias = params(cols, dtype, seed=9)
        before = (dgain.clone(), dbias.clone())
        got = M.layernorm_backward(dy, x, gain, out.mean, out.rstd, dgain=dgain, dbias=dbias,
                                   accumulate=True)
        check_backward(got, dy, f64(x), gain, out.mean, out.rstd, before)


@pytest.mark.parametrize("count", [63, 64, 65, 100, 127, 128, 129, 1023, 1024, 1025])
@pytest.mark.parametrize("rows,cols", [(40, 72), (512, 512)])
def test_numbers_of_matrices_at_the_plans_borders(count, rows, cols):
    """One wave, one block that orders the pieces, one that does not, several
    rounds of it: uneven matrices, many of one length, cut and whole, exact."""
    g = torch.Generator().manual_seed(count)
    counts = torch.randint(0, 40, (count,), generator=g)
    counts[torch.rand(count, generator=g) < 0.2] = 0
    counts[torch.rand(count, generator=g) < 0.2] = 32
    counts[count // 2], counts[-1] = 1500, 700
    off = [0] + counts.cumsum(0).tolist()
    dy = torch.randint(-9, 10, (off[-1] + 3, rows), generator=g).to(BF16).to(DEV)
    x = torch.randint(-9, 10, (off[-1] + 3, cols), generator=g).to(BF16).to(DEV)
    G = M.weight_grad(dy, M.checkpoint_save(x, "int8"), dtype=F32,
                      offsets=torch.tensor(off, dtype=torch.int64, device=DEV))
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        assert torch.equal(G[e].double(), dy[a:b].t().double() @ x[a:b].double()), e
