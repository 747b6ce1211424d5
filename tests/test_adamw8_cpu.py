"""AdamW with 8-bit states: checks that need no GPU.  The library calls fail
validation or have nothing to do, which precedes the first HIP call; the state
format is pinned by PyTorch's e4m3 and by counting."""
import ctypes
import os

import numpy as np
import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib
from oracle import adamw8_oracle as ao

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmuon.so not built")
OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
A = [0x10000000 * (i + 1) for i in range(16)]


def state(n=100, m_q=A[0], m_scale=A[1], r_q=A[2], r_scale=A[3]):
    return _lib.Adamw8State(m_q, m_scale, r_q, r_scale, n)


def step(P=A[4], G=A[5], lr=1e-3, wd=0.0, dtype=0, betas=(0.8, 0.95), eps=1e-8, t=1, count=1,
         more=(), **kw):
    # the checks of every tensor precede the first launch: a last one without
    # a gradient keeps a call that passes them from reaching the GPU
    arr = [_lib.Adamw8Tensor(P, G, state(**kw), lr, wd, 0), *more]
    c = (_lib.Adamw8Tensor * len(arr))(*arr)
    return _lib.lib().muon_adamw_byte_step_grouped(c, len(arr) if count == 1 else count, dtype,
                                               *betas, eps, t, None)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(betas=(1.0, 0.9)), ARG), (dict(betas=(0.9, -0.1)), ARG),
    (dict(betas=(float("nan"), 0.9)), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("inf")), ARG),
    (dict(t=0), ARG), (dict(count=-1), ARG), (dict(lr=float("nan")), ARG),
    (dict(wd=float("inf")), ARG), (dict(n=-1), SHAPE),
    (dict(n=_lib.MUON_ADAMW8_MAX_ELEMENTS + 1), SHAPE), (dict(P=None), ARG), (dict(G=None), ARG),
    (dict(m_q=None), ARG), (dict(r_scale=None), ARG), (dict(m_q=A[0] + 8), ARG),
    (dict(r_q=A[2] + 1), ARG), (dict(P=A[4] + 2), ARG), (dict(G=A[5] + 1, dtype=1), ARG),
    (dict(P=A[5]), ARG), (dict(m_q=A[4] + 96), ARG), (dict(m_scale=A[3]), ARG),
    # overlaps across tensors
    (dict(more=[_lib.Adamw8Tensor(A[4] + 396, A[6], state(10, A[7], A[8], A[9], A[10]), 0, 0, 0)]), ARG),
    (dict(more=[_lib.Adamw8Tensor(A[11], A[6], state(10, A[0] + 96, A[8], A[9], A[10]), 0, 0, 0)]), ARG),
    (dict(more=[_lib.Adamw8Tensor(A[11], None, state(10, A[12], A[8], A[9], A[10]), 0, 0, 0)]), ARG),
])
def test_step_refusals(kw, status):
    assert step(**kw) == status


@built
def test_nothing_to_do():
    assert step(n=0, P=None, G=None, m_q=None) == OK
    assert _lib.lib().muon_adamw_byte_step_grouped(None, 0, 0, 0.9, 0.9, 1e-8, 1, None) == OK
    assert _lib.lib().muon_adamw_byte_step_grouped(None, 1, 0, 0.9, 0.9, 1e-8, 1, None) == ARG
    assert _lib.lib().muon_adamw_byte_moments(None, 0, None, None, 0, None) == OK
    empty = (_lib.Adamw8State * 1)(state(0, None, None, None, None))
    assert _lib.lib().muon_adamw_byte_moments(empty, 1, None, None, 1, None) == OK


@built
@pytest.mark.parametrize("kw,m,r,dtype,status", [
    ({}, A[6], A[7], 5, DTYPE), ({}, None, A[7], 0, ARG), ({}, A[6], None, 0, ARG),
    ({}, A[6] + 2, A[7], 0, ARG), ({}, A[6], A[6] + 396, 0, ARG), ({}, A[0], A[7], 0, ARG),
    ({}, A[6], A[3], 0, ARG), (dict(n=-5), A[6], A[7], 0, SHAPE), (dict(m_q=A[0] + 4), A[6], A[7], 0, ARG),
])
def test_moments_refusals(kw, m, r, dtype, status):
    arr = (_lib.Adamw8State * 1)(state(**kw))
    assert _lib.lib().muon_adamw_byte_moments(arr, 1, m, r, dtype, None) == status
    assert _lib.lib().muon_adamw_byte_moments(arr, -1, A[6], A[7], 0, None) == ARG


def test_front_end_refusals():
    cpu = [torch.zeros(32).to(torch.float8_e4m3fn), torch.zeros(1, dtype=torch.uint8),
           torch.zeros(32, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8)]
    with pytest.raises(ValueError, match="GPU"):
        M.AdamwState8(*cpu, 32)
    with pytest.raises(ValueError):
        M.AdamwState8(*cpu, -1)
    with pytest.raises(TypeError):
        M.adamw8_tensor(torch.zeros(3), torch.zeros(3), None, lr=0.1)
    with pytest.raises(ValueError):
        M.adamw8_moments([])
    with pytest.raises(TypeError):
        M.adamw8_step_grouped([], torch.float16, step=1)
    with pytest.raises(ValueError, match="states"):
        M.AdamWStep([], states="4bit")


def test_struct_layout():
    assert ctypes.sizeof(_lib.Adamw8State) == 40
    assert ctypes.sizeof(_lib.Adamw8Tensor) == 80


# ------------------------------------------------------------------ the format
def test_m_numbers_are_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ao.numbers("m"), want, equal_nan=True)


def test_r_numbers():
    v = ao.numbers("r")
    assert v[0] == 0 and v[1] == 2.0 ** -10 and v[15] == 15 * 2.0 ** -10 and v[16] == 2.0 ** -6
    assert v[255] == 496 and (np.diff(v) > 0).all()
    assert ((v[17:] - v[16:-1]) / v[16:-1] <= 2.0 ** -4).all()


@pytest.mark.parametrize("which", ["m", "r"])
def test_kept_numbers_are_the_neighbours_and_unbiased(which):
    """Each element is kept as the number below or above, up as often as its
    distance says: the mean over 65536 shares of a step is the element."""
    top = ao.FORMATS[which][0]
    a = np.array([1.03, 0.013, 0.3, top, 2.0 ** -9 * 0.3, 17.77, top * 0.999])
    scale = np.array([127])
    u = (np.arange(65536) + 0.5) / 65536
    v = np.stack([ao.kept(a, scale, s, which) for s in u[::64]])
    assert np.isin(v, ao.numbers(which)).all()
    if which == "r":
        assert (v > 0).all()       # a root that is not zero stays so
        a, v = np.delete(a, 4), np.delete(v, 4, axis=1)
    grid = np.sort(ao.numbers(which)[~np.isnan(ao.numbers(which))])
    below = grid[np.searchsorted(grid, a, side="right") - 1]
    above = grid[np.minimum(np.searchsorted(grid, a, side="left"), grid.size - 1)]
    assert ((v == below) | (v == above)).all()
    assert np.allclose(v.mean(0), a, rtol=0, atol=(above - below).max() / 1024 + 1e-12)


def test_exact_numbers_are_kept():
    for which in "mr":
        v = ao.numbers(which)
        v = v[np.isfinite(v)]
        for s in (0.5 / 65536, 1 - 0.5 / 65536):
            got = ao.kept(v, np.full(-(-v.size // 32), 127), np.full(v.size, s), which)
            assert np.array_equal(got, v)


def test_the_rounding_follows_a_slow_average():
    """A root that decays by 0.0005 a step, far below half a step of the format,
    follows its formula; rounding to nearest would leave it where it is."""
    n, r = 4096, np.full(4096, 1.3)
    for t in range(400):
        r = np.sqrt(0.999 * r * r)
        r = ao.kept(r, np.full(n // 32, 127), ao.share(n, 1000 + 77 * t, "r"), "r")
    # a random walk of 400 steps of at most 1/16 each: its mean over 4096
    # elements is off by less than 6 / 16 * sqrt(400 / 4096) = 0.12
    want = 1.3 * 0.999 ** 200
    assert abs(r.mean() - want) < 0.12 and r.std() > 0
    near = np.sqrt(0.999 * 1.3125 ** 2)
    assert ao.kept(np.array([near]), np.array([127]), np.array([0.5]), "r")[0] == 1.3125


def test_random_bits_differ_between_elements_seeds_and_halves():
    a, b = ao.random_bits(1 << 16, 1), ao.random_bits(1 << 16, 2)
    assert np.unique(a).size == a.size          # the mixing is one to one
    assert (a != b).all() or (a == b).mean() < 1e-3
    for x in (a >> 16, a & 0xffff):
        assert abs(x.mean() / 65535 - 0.5) < 5 / np.sqrt(12 * x.size)
    assert abs(np.corrcoef(a >> 16, a & 0xffff)[0, 1]) < 0.02


def test_random_bits_of_parameters_and_steps_share_no_run():
    """The optimizer's seeds of 64 parameters and steps: no tensor's random bits are
    another's, shifted.  2^18 draws of 2^32 numbers repeat 2^36 / 2^33 = 8 times by
    chance; a shifted run would repeat some 4000 times."""
    opt = object.__new__(M.AdamWStep)
    opt.seed, opt.entries = 3, [None] * 16
    seeds = []
    for opt.step_count in range(1, 5):
        seeds += [opt._seed(i) for i in range(16)]
    assert len(set(seeds)) == 64 and all(0 <= s < 1 << 32 for s in seeds)
    bits = np.concatenate([ao.random_bits(4096, s) for s in seeds])
    assert bits.size - np.unique(bits).size < 64


@pytest.mark.parametrize("field", ["m_q", "m_scale", "r_q", "r_scale", "n", "device"])
def test_a_states_fields_are_not_assigned(field):
    """The library steps the tensors that a state was made of: another one put in
    their place would be neither read nor kept alive."""
    with pytest.raises(AttributeError):
        setattr(object.__new__(M.AdamwState8), field, torch.zeros(32))


@built
@pytest.mark.parametrize("count", [(1 << 40) + 1, 1 << 60, 1 << 62, (1 << 63) - 1])
def test_counts_that_no_host_can_list(count):
    """Refused before a tensor is looked at, with no C++ exception on the way."""
    L, p = _lib.lib(), ctypes.c_void_p
    one = (_lib.Adamw8Tensor * 1)()
    assert L.muon_adamw_byte_step_grouped(one, count, 0, 0.8, 0.95, 1e-8, 1, None) == ARG
    assert L.muon_adamw_byte_moments((_lib.Adamw8State * 1)(), count, p(A[6]), p(A[7]), 0, None) == ARG
    assert L.muon_adamw_step_grouped((_lib.AdamwTensor * 1)(), count, 0, 0.8, 0.95, 1e-8, 1, None) == ARG
