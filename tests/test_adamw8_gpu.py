"""AdamW with 8-bit states on the GPU against the fp64 oracle.

The kernel computes m' and r' in float32 and rounds each to 8 bits by known
random bits.  With d the most that float32 can be off, the kept number must lie
between what is kept of the oracle's value minus d and plus d: rounding down
after an addition is monotone.  u = 2^-24 is half a step of float32:
  m' = b1 m + (1 - b1) g: each product has two rounded factors or results
       (2 u), the sum one more: d = 3 u (|b1 m| + |(1 - b1) g|)
  r' : each of the two terms under the root has three roundings (4 with the
       sum), the root halves them and adds one: d = 3 u r'
  p' : m' / (r' s + eps): 3 + 1 u for m' relative to its terms, 3 + 3 u for the
       denominator, 1 each for the division, step size (2), decay and sum
"""
import copy

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib
from oracle import adamw8_oracle as ao

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BETAS, EPS = (0.8, 0.95), 1e-10


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(n, dtype, seed, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    P = (0.02 * torch.randn(n, generator=g)).to(dtype).to(DEV)
    s = torch.exp(torch.randn((n + 15) // 16, generator=g)).repeat_interleave(16)[:n]
    G = (size * s * torch.randn(n, generator=g)).to(dtype).to(DEV)
    return P, G


def values(st):
    out = []
    for which, q, scale in (("m", st.m_q.view(torch.uint8), st.m_scale), ("r", st.r_q, st.r_scale)):
        out.append(ao.values(q.cpu().numpy(), scale.cpu().numpy(), st.n, which))
    return out


def check(before, P, G, st, *, lr, wd, step, seed, betas=BETAS, eps=EPS):
    """One step from ``before`` (P, m, r as float64) against the oracle."""
    p0, m0, r0 = before
    g, n = f64(G), P.numel()
    p, m, r = ao.step(p0, g, m0, r0, lr=lr, beta1=betas[0], beta2=betas[1], eps=eps,
                      weight_decay=wd, step=step)
    terms = np.abs(betas[0] * m0) + np.abs((1 - betas[0]) * g)
    d_m, d_r = 3.01 * U * terms, 3.01 * U * r
    for which, x, d, q, scale in (("m", m, d_m, st.m_q.view(torch.uint8), st.m_scale),
                                  ("r", r, d_r, st.r_q, st.r_scale)):
        q, scale = q.cpu().numpy(), scale.cpu().numpy().astype(np.int64)
        away = np.maximum(np.abs(x) - d, 0)
        assert (scale >= ao.scale_bytes(away, which)).all(), which
        assert (scale <= ao.scale_bytes(np.abs(x) + d, which)).all(), which
        assert not q.reshape(-1)[n:].any()
        added = ao.share(n, seed, which)
        got = np.abs(ao.values(q, scale, n, which))
        lo, hi = ao.kept(away, scale, added, which), ao.kept(np.abs(x) + d, scale, added, which)
        assert (got >= lo).all() and (got <= hi).all(), which
        sign = ao.values(q, scale, n, which)
        assert (np.sign(sign)[np.abs(x) > d] * np.sign(x)[np.abs(x) > d] >= 0).all()
    # P
    bc1, bc2 = 1 - betas[0] ** step, 1 - betas[1] ** step
    denom = r / np.sqrt(bc2) + eps
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(denom > 0, np.abs(m) / denom, 0)
        d_ratio = np.where(denom > 0, d_m / denom, 0) + 8 * U * ratio
    bound = abs(lr) / bc1 * (d_ratio + 3 * U * ratio) + 3 * U * np.abs(p0) + U * np.abs(p)
    bound = bound * 1.01 + HALF[P.dtype] * (np.abs(p) + bound)
    assert (np.abs(f64(P) - p) <= bound).all(), np.max(np.abs(f64(P) - p) - bound)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 31, 32, 33, 255, 777, 4096, 4097, 8191, 100_003])
def test_steps_against_oracle(n, dtype):
    P, G = draw(n, dtype, n)
    st = M.AdamwState8.zeros(n, DEV)
    assert st.nbytes == 2 * ((n + 31) // 32) * 33
    for t in (1, 2, 3):
        before = (f64(P), *values(st))
        M.adamw8_step(P, G, st, lr=0.015, step=t, seed=99 * t, weight_decay=0.1)
        torch.cuda.synchronize()
        check(before, P, G, st, lr=0.015, wd=0.1, step=t, seed=99 * t)
        _, G = draw(n, dtype, n + 1000 * t, 3e-3)


@pytest.mark.parametrize("betas,eps,lr", [((0.0, 0.0), 1e-8, 0.1), ((0.9, 0.999), 1e-8, 3e-4),
                                          ((0.95, 0.95), 0.0, -0.1), ((0.8, 0.95), 1.0, 0.0)])
def test_scalars(betas, eps, lr):
    P, G = draw(5000, torch.float32, 5)
    st = M.AdamwState8.zeros(5000, DEV)
    for t in (1, 2):
        before = (f64(P), *values(st))
        M.adamw8_step(P, G, st, lr=lr, step=t, seed=t, betas=betas, eps=eps, weight_decay=0.0)
        check(before, P, G, st, lr=lr, wd=0.0, step=t, seed=t, betas=betas, eps=eps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [1, 3, 7])
def test_unaligned_parameters(dtype, shift):
    """P and G at any element: equal bits to the aligned call, and nothing
    around them is written."""
    n = 5003
    P, G = draw(n, dtype, 11)
    Pb, Gb = torch.full((n + 16,), 7.0, dtype=dtype, device=DEV), torch.zeros(n + 16, dtype=dtype, device=DEV)
    Pb[shift:shift + n] = P
    Gb[shift:shift + n] = G
    a, b = M.AdamwState8.zeros(n, DEV), M.AdamwState8.zeros(n, DEV)
    for t in (1, 2):
        M.adamw8_step(P, G, a, lr=0.01, step=t, seed=t)
        M.adamw8_step(Pb[shift:shift + n], Gb[shift:shift + n], b, lr=0.01, step=t, seed=t)
    assert torch.equal(P, Pb[shift:shift + n])
    assert bool((Pb[:shift] == 7).all()) and bool((Pb[shift + n:] == 7).all())
    for k in ("m_q", "m_scale", "r_q", "r_scale"):
        assert torch.equal(getattr(a, k).view(torch.uint8), getattr(b, k).view(torch.uint8)), k


def test_grouped_equals_single_and_moments():
    """100 tensors (80 not empty: two launches), each with its own lr, decay and seed, some
    empty: bits of one call per tensor; the moments come back one behind the
    other, exactly."""
    sizes = [1, 0, 64, 777, 4096, 5000, 12345, 33, 0, 8192] * 10
    one, many = [], []
    for i, n in enumerate(sizes):
        P, G = draw(n, torch.bfloat16, 50 + i)
        one.append((P, G, M.AdamwState8.zeros(n, DEV)))
        many.append((P.clone(), G, M.AdamwState8.zeros(n, DEV)))
    for t in (1, 2):
        M.adamw8_step_grouped([M.adamw8_tensor(*x, lr=0.01 * (i % 3), weight_decay=0.1 * (i % 2), seed=i + 1000 * t)
                               for i, x in enumerate(many)], torch.bfloat16, step=t)
        for i, x in enumerate(one):
            M.adamw8_step(*x, lr=0.01 * (i % 3), weight_decay=0.1 * (i % 2), seed=i + 1000 * t, step=t)
    for dtype in (torch.float32, torch.bfloat16):
        m, r = M.adamw8_moments([x[2] for x in many], dtype)
        assert m.dtype == r.dtype == dtype and m.numel() == r.numel() == sum(sizes)
        want = [np.concatenate([values(x[2])[k] for x in one]) for k in (0, 1)]
        assert np.array_equal(f64(m), want[0]) and np.array_equal(f64(r), want[1])
    assert all(torch.equal(a[0], b[0]) for a, b in zip(one, many))


def test_same_seed_same_bits_other_seed_others():
    outs = []
    for seed in (3, 3, 4):
        P, G = draw(70_000, torch.bfloat16, 15)
        st = M.AdamwState8.zeros(70_000, DEV)
        M.adamw8_step(P, G, st, lr=0.004, step=1, seed=seed)
        outs.append((P, st.m_q.view(torch.uint8), st.r_q))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    assert torch.equal(outs[0][0], outs[2][0])          # P is made before the rounding
    assert (outs[0][1] != outs[2][1]).float().mean() > 0.1
    assert (outs[0][2] != outs[2][2]).float().mean() > 0.1


def test_indices_past_32_bits_of_elements():
    """The last elements of a tensor of more than 2^32: their random bits use
    the upper half of the index."""
    n = (1 << 32) + 4096 + 40
    P = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    G = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    st = M.AdamwState8.zeros(n, DEV)
    tail = slice(n - 5000, n)
    _, g = draw(5000, torch.bfloat16, 21)
    G[tail] = g
    M.adamw8_step(P, G, st, lr=0.01, step=1, seed=5, weight_decay=0.0)
    i = np.arange(n - 5000, n, dtype=np.uint64)
    low = np.uint64(0xffffffff)
    x = ((i & low) * np.uint64(0x9e3779b1) + (i >> np.uint64(32)) * np.uint64(0x85ebca77) + np.uint64(5)) & low
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7feb352d)) & low
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846ca68b)) & low
    added = (((x ^ (x >> np.uint64(16))) >> np.uint64(16)).astype(np.float64) + 0.5) / 65536
    m = 0.2 * f64(g)
    first = (n - 5000) // 32 * 32
    skip = n - 5000 - first
    scale = st.m_scale[first // 32:].cpu().numpy()
    pad = np.concatenate([np.zeros(skip), m])
    padded = np.concatenate([np.zeros(skip), added])
    q = st.m_q[first:].view(torch.uint8).cpu().numpy()
    got = np.abs(ao.values(q, scale, pad.size, "m"))
    lo = ao.kept(np.abs(pad) * (1 - 4 * U), scale, padded, "m")
    hi = ao.kept(np.abs(pad) * (1 + 4 * U), scale, padded, "m")
    assert (got >= lo).all() and (got <= hi).all()
    assert not P[:4096].any() and bool((P[tail] != 0).any())


def test_zero_gradients_and_states():
    P, _ = draw(1000, torch.float32, 12)
    P0 = P.clone()
    st = M.AdamwState8.zeros(1000, DEV)
    M.adamw8_step(P, torch.zeros_like(P), st, lr=0.7, step=5, weight_decay=1e-3)
    assert not st.m_q.view(torch.uint8).any() and not st.r_q.any()
    assert torch.equal(P, P0 * float(np.float32(1 - 0.7e-3)))


def test_a_root_is_never_lost():
    """Elements far below their block's largest: their root is kept as the
    smallest number, so that the next step of a zero gradient stays bounded."""
    G = torch.full((64,), 1e-12, device=DEV)
    G[0], G[32] = 1.0, 1e5
    P, st = torch.zeros(64, device=DEV), M.AdamwState8.zeros(64, DEV)
    M.adamw8_step(P, G, st, lr=0.1, step=1)
    m, r = M.adamw8_moments(st)
    assert bool((r > 0).all())
    before = P.clone()
    M.adamw8_step(P, torch.zeros_like(G), st, lr=0.1, step=2)
    assert float((P - before).abs().max()) <= 0.1 * 2


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_gradients_mark_their_block(bad):
    n = 5000
    P, G = draw(n, torch.bfloat16, 13)
    G[70] = bad
    st = M.AdamwState8.zeros(n, DEV)
    P0 = P.clone()
    M.adamw8_step(P, G, st, lr=0.015, step=2)
    m, r = M.adamw8_moments([st])
    hit = torch.zeros(n, dtype=torch.bool, device=DEV)
    hit[64:96] = True
    assert torch.equal(torch.isnan(m), hit) and torch.equal(torch.isnan(r), hit)
    assert bool(torch.isnan(P[70])) and bool(torch.isfinite(P[:70]).all()) and bool(torch.isfinite(P[71:]).all())
    assert not torch.equal(P, P0)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15, 1e18])
def test_ends_of_float32(size):
    """Gradients whose squares come near float32's ends or leave it: finite
    parameters and m.  g * g is infinite in float32 where |g| >= 2^64 (2^128 is
    the first number behind float32's range, and nothing below 2^64 in float32
    has a square that rounds to it): r is then infinite, and its block marked."""
    P, G = draw(4096, torch.float32, 31, size)
    st = M.AdamwState8.zeros(4096, DEV)
    M.adamw8_step(P, G, st, lr=1e-3, step=1, eps=1e-30)
    m, r = M.adamw8_moments(st)
    assert bool(torch.isfinite(P).all()) and bool(torch.isfinite(m).all())
    out = (G.abs() >= 2.0 ** 64).view(-1, 32).any(1).repeat_interleave(32)
    assert torch.equal(torch.isnan(r), out) and bool(out.any()) == (size == 1e18)
    want = 0.2 * f64(G)
    scale = st.m_scale.cpu().numpy()
    lo = ao.kept(np.abs(want) * (1 - 4 * U), scale, ao.share(4096, 0, "m"), "m")
    hi = ao.kept(np.abs(want) * (1 + 4 * U), scale, ao.share(4096, 0, "m"), "m")
    assert (np.abs(f64(m)) >= lo).all() and (np.abs(f64(m)) <= hi).all()


def test_a_stream_of_its_own_and_a_graph():
    """On another stream, and captured: the replays are the eager steps."""
    n = 30_000
    P, G = draw(n, torch.bfloat16, 41)
    ref, rst = P.clone(), M.AdamwState8.zeros(n, DEV)
    st = M.AdamwState8.zeros(n, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.adamw8_step(P, G, st, lr=0.01, step=1, seed=7, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    M.adamw8_step(ref, G, rst, lr=0.01, step=1, seed=7)
    assert torch.equal(P, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.adamw8_step(P, G, st, lr=0.01, step=2, seed=8)
    for k in range(3):
        graph.replay()
        G.mul_(2)      # exact, and taken back
        torch.cuda.synchronize()
        G.div_(2)
        M.adamw8_step(ref, G, rst, lr=0.01, step=2, seed=8)
        assert torch.equal(P, ref) and torch.equal(st.r_q, rst.r_q), k


def test_optimizer_front_end():
    """AdamWStep(states="8bit") steps each parameter as the single calls do, with
    seeds that differ between parameters and steps, and through the hybrid."""
    torch.manual_seed(3)
    shapes = [(300, 96), (96,), (7, 5, 3)]
    params = [torch.nn.Parameter((torch.randn(s) * 0.02).to(DEV)) for s in shapes]
    params.append(torch.nn.Parameter((torch.randn(100) * 0.02).to(torch.bfloat16).to(DEV)))
    hidden = torch.nn.Parameter((torch.randn(64, 96) * 0.02).to(DEV))
    opt = M.HybridMuonAdamW([hidden], [dict(params=params[:2], lr=0.1), dict(params=params[2:], lr=0.01, weight_decay=0.0)],
                            adamw_kwargs=dict(states="8bit", seed=5))
    copies = [p.detach().clone() for p in params]
    states = [M.AdamwState8.zeros(p.numel(), DEV) for p in params]
    seen = set()
    for t in (1, 2, 3):
        for p in params + [hidden]:
            p.grad = torch.randn_like(p) * 1e-3
        opt.step()
        for i, (c, p, s) in enumerate(zip(copies, params, states)):
            seed = opt.adamw._seed(i)
            seen.add(seed)
            M.adamw8_step(c, p.grad, s, lr=0.1 if i < 2 else 0.01, step=t, seed=seed,
                          weight_decay=M.AUX_WEIGHT_DECAY if i < 2 else 0.0)
            assert torch.equal(c, p.detach()), (t, i)
    assert len(seen) == 12
    other = copy.deepcopy(opt.adamw.states[0])
    assert torch.equal(other.r_q, states[0].r_q) and other.r_q.data_ptr() != states[0].r_q.data_ptr()


def test_follows_the_float32_optimizer():
    """200 steps on noisy gradients with a drift: the parameters end where
    float32 states put them, to a few percent of the way."""
    n = 20_000
    g = torch.Generator().manual_seed(1)
    drift = 1e-3 * torch.randn(n, generator=g).to(DEV)
    P8, P32 = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    st = M.AdamwState8.zeros(n, DEV)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    for t in range(1, 201):
        G = drift + 1e-3 * torch.randn(n, generator=g).to(DEV)
        M.adamw8_step(P8, G, st, lr=1e-3, step=t, seed=t * 7919, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)
        M.adamw_step(P32, G, m, v, lr=1e-3, step=t, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)
    a, b = f64(P8), f64(P32)
    assert np.linalg.norm(a - b) < 0.1 * np.linalg.norm(b)


def test_gpu_front_end_refusals():
    st = M.AdamwState8.zeros(10, DEV)
    P = torch.zeros(10, device=DEV)
    with pytest.raises(ValueError):
        M.adamw8_tensor(torch.zeros(9, device=DEV), P, st, lr=0.1)
    with pytest.raises(TypeError):
        M.adamw8_tensor(P, P.bfloat16(), st, lr=0.1)
    with pytest.raises(TypeError):
        M.adamw8_tensor(P.half(), P.half(), st, lr=0.1)
    with pytest.raises(ValueError):
        M.AdamwState8(st.m_q, st.m_scale, st.r_q, st.r_scale, 33)
    with pytest.raises(TypeError):
        M.AdamwState8(st.r_q, st.m_scale, st.r_q, st.r_scale, 10)
    with pytest.raises(M.MuonError):      # the same buffer twice
        M.adamw8_step(P, P, st, lr=0.1, step=1)
    assert _lib.MUON_ADAMW8_TENSORS_PER_LAUNCH == 56


def test_restoring_a_state():
    """A state takes a saved one's values into its tensors, or a new state is made
    of the saved tensors; both go on as the saved one does.  Assignment is refused;
    a shallow copy shares the tensors, a deep one has its own."""
    n = 1000
    P, G = draw(n, torch.float32, 1)
    st = M.AdamwState8.zeros(n, DEV)
    M.adamw8_step(P, G, st, lr=0.01, step=1, seed=1)
    saved = [t.clone() for t in (st.m_q, st.m_scale, st.r_q, st.r_scale)]
    deep, shallow, p = copy.deepcopy(st), copy.copy(st), P.clone()
    M.adamw8_step(P, G, st, lr=0.01, step=2, seed=2)
    want = values(st)
    filled, made = M.AdamwState8.zeros(n, DEV), M.AdamwState8(*saved, n)
    for name, t in zip(("m_q", "m_scale", "r_q", "r_scale"), saved):
        with pytest.raises(AttributeError):
            setattr(filled, name, t)
        getattr(filled, name).copy_(t)
    for state in (filled, made, deep):
        q = p.clone()
        M.adamw8_step(q, G, state, lr=0.01, step=2, seed=2)
        assert torch.equal(q, P)
        assert all(np.array_equal(a, b) for a, b in zip(values(state), want))
    assert shallow.m_q.data_ptr() == st.m_q.data_ptr() and shallow.n == n and shallow.device == st.device
    assert all(np.array_equal(a, b) for a, b in zip(values(shallow), want))
