"""C ABI and binding checks of the layer operators that need no GPU: every call
here fails validation, which precedes the first HIP call."""
import ctypes
import os

import pytest
import torch

import muon_step_03_amd as M
from muon_step_03_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmuon.so not built")

F32, BF16 = _lib.MUON_DTYPE_F32, _lib.MUON_DTYPE_BF16
# Fake device addresses, far apart: never dereferenced.
A = [0x10000000 * (i + 1) for i in range(12)]
OK, ARG, SHAPE, DTYPE, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def ckpt(q=A[8], scale=A[9], tokens=16, cols=64, fmt=0):
    return ctypes.byref(_lib.Ckpt(q, scale, tokens, cols, fmt))


def save(L, x=A[0], ldx=64, dtype=F32, ck=None):
    return L.muon_checkpoint_save(x, ldx, dtype, ck if ck is not None else ckpt(), None)


CKPT_FAULTS = [
    (dict(fmt=2), ARG), (dict(fmt=-1), ARG), (dict(q=None), ARG), (dict(scale=None), ARG),
    (dict(q=A[8] + 8), ARG), (dict(scale=A[9] + 2), ARG), (dict(tokens=-1), SHAPE),
    (dict(tokens=_lib.MUON_MAX_TOKENS + 1), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=_lib.MUON_MAX_DIM + 1), SHAPE),
]


@pytest.mark.parametrize("fault,status", CKPT_FAULTS)
def test_checkpoint_descriptor(L, fault, status):
    assert save(L, ck=ckpt(**fault)) == status
    assert L.muon_checkpoint_restore(ckpt(**fault), A[0], F32, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), DTYPE), (dict(x=None), ARG), (dict(x=A[0] + 2), ARG), (dict(ldx=63), ARG),
    (dict(ldx=(1 << 24) + 1), ARG), (dict(x=A[8]), ARG), (dict(x=A[9] - 4), ARG),
])
def test_checkpoint_save_refusals(L, kw, status):
    assert save(L, **kw) == status


def test_checkpoint_null_descriptor_and_empty(L):
    assert L.muon_checkpoint_save(A[0], 64, F32, None, None) == ARG
    assert L.muon_checkpoint_restore(None, A[0], F32, None) == ARG
    assert L.muon_checkpoint_restore(ckpt(), None, F32, None) == ARG
    assert L.muon_checkpoint_restore(ckpt(), A[0], 5, None) == DTYPE
    empty = ckpt(q=None, scale=None, tokens=0)
    assert L.muon_checkpoint_save(None, 64, F32, empty, None) == OK
    assert L.muon_checkpoint_restore(empty, None, F32, None) == OK


def forward(L, x=A[0], ldx=64, gain=A[1], bias=A[2], tokens=16, cols=64, dtype=F32, pdtype=F32,
            eps=1e-5, y=A[3], mean=A[4], rstd=A[5], xc=None, yc=None):
    return L.muon_layernorm_forward(x, ldx, gain, bias, tokens, cols, dtype, pdtype, eps, y, mean,
                                    rstd, xc, yc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(pdtype=-1), DTYPE), (dict(tokens=-1), SHAPE),
    (dict(tokens=_lib.MUON_MAX_TOKENS + 1), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=_lib.MUON_MAX_DIM + 1, ldx=1 << 20), SHAPE), (dict(eps=-1e-9), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(x=None), ARG),
    (dict(gain=None), ARG), (dict(y=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG),
    (dict(ldx=60), ARG), (dict(x=A[0] + 1), ARG), (dict(mean=A[4] + 2), ARG),
    (dict(y=A[0]), ARG), (dict(y=A[0] + 4095), ARG), (dict(mean=A[5]), ARG), (dict(y=A[2]), ARG),
    (dict(gain=A[3] + 128), ARG),
])
def test_forward_refusals(L, kw, status):
    assert forward(L, **kw) == status


@pytest.mark.parametrize("which", ["xc", "yc"])
@pytest.mark.parametrize("fault,status", CKPT_FAULTS + [(dict(tokens=15), SHAPE),
                                                        (dict(cols=63), SHAPE),
                                                        (dict(q=A[3]), ARG),
                                                        (dict(scale=A[0] + 16), ARG)])
def test_forward_checkpoints(L, which, fault, status):
    assert forward(L, **{which: ckpt(**fault)}) == status


def test_forward_two_checkpoints_in_one_place(L):
    assert forward(L, xc=ckpt(), yc=ckpt()) == ARG


def test_forward_no_tokens(L):
    assert forward(L, tokens=0, x=None, y=None, mean=None, rstd=None) == OK


def backward(L, dy=A[0], lddy=64, x=A[1], ldx=64, xc=None, gain=A[2], mean=A[3], rstd=A[4],
             tokens=1000, cols=64, dtype=F32, pdtype=F32, dx=A[5], dgain=A[6], dbias=A[7], acc=0,
             ws=A[10], wsb=1 << 20):
    return L.muon_layernorm_backward(dy, lddy, x, ldx, xc, gain, mean, rstd, tokens, cols, dtype,
                                     pdtype, dx, dgain, dbias, acc, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(pdtype=3), DTYPE), (dict(tokens=-5), SHAPE),
    (dict(cols=0), SHAPE), (dict(dy=None), ARG), (dict(x=None), ARG), (dict(gain=None), ARG),
    (dict(mean=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG), (dict(dgain=None), ARG),
    (dict(lddy=63), ARG), (dict(ldx=0), ARG), (dict(ws=None), ARG), (dict(wsb=16), WS),
    (dict(dx=A[0]), ARG), (dict(dx=A[1] + 8), ARG), (dict(dgain=A[7]), ARG),
    (dict(dbias=A[2] + 4), ARG), (dict(ws=A[5] - 16), ARG), (dict(ws=A[0], tokens=16), ARG), (dict(dx=A[5] + 2), ARG),
])
def test_backward_refusals(L, kw, status):
    assert backward(L, **kw) == status


def test_backward_source_is_one_of_two(L):
    assert backward(L, xc=ckpt(tokens=1000)) == ARG            # both
    assert backward(L, x=None, xc=ckpt(cols=32)) == SHAPE
    assert backward(L, x=None, xc=ckpt(tokens=1000), dx=A[9]) == ARG


def test_backward_no_tokens_accumulating(L):
    assert backward(L, tokens=0, dy=None, x=None, dx=None, mean=None, rstd=None, acc=1) == OK


def weight(L, dy=A[0], lddy=96, dtype=F32, x=None, offsets=None, count=1, rows=96, G=A[2],
           gdtype=F32, acc=0, ws=A[4], wsb=1 << 26):
    x = x if x is not None else ckpt(tokens=4000)
    return L.muon_weight_grad(dy, lddy, dtype, x, offsets, count,
                              rows, G, gdtype, acc, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(gdtype=2), DTYPE), (dict(count=-1), ARG), (dict(rows=0), SHAPE),
    (dict(rows=_lib.MUON_MAX_DIM + 1, lddy=1 << 20), SHAPE), (dict(count=2), ARG),
    (dict(count=1 << 40, offsets=A[5]), SHAPE), (dict(count=1 << 23, offsets=0x6000_0000_0000, G=0x7000_0000_0000), SHAPE),
    (dict(dy=None), ARG), (dict(G=None), ARG), (dict(ws=None), ARG), (dict(lddy=95), ARG),
    (dict(dy=A[0] + 2), ARG), (dict(offsets=A[5] + 4), ARG), (dict(G=A[0]), ARG),
    (dict(G=A[8] + 64), ARG), (dict(G=A[5], offsets=A[5]), ARG), (dict(ws=A[2]), ARG),
    (dict(wsb=8), WS),
])
def test_weight_grad_refusals(L, kw, status):
    assert weight(L, **kw) == status


@pytest.mark.parametrize("fault,status", CKPT_FAULTS)
def test_weight_grad_checkpoint(L, fault, status):
    assert weight(L, x=ckpt(**fault)) == status


def test_weight_grad_nothing_to_do(L):
    assert weight(L, count=0, G=None, ws=None) == OK
    assert weight(L, x=ckpt(q=None, scale=None, tokens=0), dy=None, acc=1) == OK


def test_workspace_sizes(L):
    assert L.muon_layernorm_workspace_bytes(-1, 5) == 0
    assert L.muon_layernorm_workspace_bytes(5, 0) == 0
    # one block's rows need no partial sums
    assert L.muon_layernorm_workspace_bytes(0, 64) == 0
    assert L.muon_layernorm_workspace_bytes(12, 768) == 0
    # partial sums grow with the tokens up to a fixed number of blocks
    big = L.muon_layernorm_workspace_bytes(1 << 20, 1024)
    assert big == L.muon_layernorm_workspace_bytes(1 << 30, 1024) > 1024 * 8
    assert L.muon_weight_grad_workspace_bytes(0, 0, 5, 5, 5, 0) == 0
    assert L.muon_weight_grad_workspace_bytes(1, 0, 5, 0, 5, 0) == 0
    assert L.muon_weight_grad_workspace_bytes(1, 0, -1, 5, 5, 0) == 0
    assert L.muon_weight_grad_workspace_bytes(1, 0, 5, 5, _lib.MUON_MAX_DIM + 1, 0) == 0
    assert L.muon_weight_grad_workspace_bytes(1, 0, 5, 5, 5, 2) == 0
    # one piece, nothing to repack
    assert L.muon_weight_grad_workspace_bytes(1, 0, 96, 768, 768, BF16) == 0
    # partial sums and a table entry for each piece of at least 128 tokens,
    # and dy once more in three bf16 parts (float32) or in padded rows
    for count, tokens, rows, cols in [(1, 1 << 20, 64, 64), (64, 49152, 1408, 512),
                                      (1, 16384, 4096, 1024), (7, 100, 33, 1000),
                                      (1, 65536, 1001, 777)]:
        for dtype, part in ((F32, 6), (BF16, 0 if rows % 8 == 0 else 2)):
            got = L.muon_weight_grad_workspace_bytes(count, 1, tokens, rows, cols, dtype)
            pieces = tokens // 128 + count
            most = pieces * (rows * cols * 4 + 48) + (rows + 7) * tokens * part + 1024
            assert 256 <= got <= most


def test_layers_refuse_mismatched_arguments():
    x, W = torch.zeros(4, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="2-D"):
        M.linear(x, W[0])
    with pytest.raises(TypeError, match="dtype"):
        M.linear(x, W.bfloat16())
    with pytest.raises(ValueError, match="columns"):
        M.linear(x, W[:, :32])
    with pytest.raises(ValueError, match="on a GPU"):
        M.linear(x, W.clone().requires_grad_())
    with pytest.raises(ValueError, match="on a GPU"):
        M.layer_norm(x, W[0])


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 64)
    v = torch.zeros(64)
    with pytest.raises(ValueError, match="on a GPU"):
        M.layernorm_forward(x, v)
    with pytest.raises(ValueError, match="on a GPU"):
        M.checkpoint_save(x)
    with pytest.raises(ValueError, match="on a GPU"):
        M.layernorm_backward(x, x, v, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="on a GPU"):
        M.weight_grad(x, None)
    with pytest.raises(ValueError, match="2-D"):
        M.layernorm_forward(x[0], v)
    with pytest.raises(TypeError, match="torch.Tensor"):
        M.checkpoint_save([1.0])
    with pytest.raises(TypeError, match="ActCheckpoint"):
        M.checkpoint_restore(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.ActCheckpoint(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(TypeError, match="float8_e4m3fn or int8"):
        M.ActCheckpoint(x, torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="format"):
        M.ActCheckpoint.empty(4, 64, "e5m2", device="cpu")


def test_few_long_rows_are_not_left_to_one_block(L):
    """One block of the norm's backward pass needs no workspace.  Rows of more
    than 4096 columns are one pass each: a few of 8192, one of 32768."""
    one = {4096: 16, 5632: 3, 8192: 3, 8193: 2, 16384: 2, 16385: 1, 32768: 1}
    for cols, rows in one.items():
        assert L.muon_layernorm_workspace_bytes(rows, cols) == 0, cols
        assert L.muon_layernorm_workspace_bytes(rows + 1, cols) > 0, cols
