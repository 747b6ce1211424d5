"""Inputs, oracles and error bounds shared by the tests of the linear products
(not collected by pytest).

u = 2^-24 is half a step of float32.  A product of two bf16 numbers is exact in
float32, one of two float32 numbers off by u; a sum of k terms in any order by
(k - 1) u of the sum of magnitudes (first order; 8 u more cover that).  A result
in bfloat16 is rounded once, by at most 2^-8 of itself.

8-bit operands with a bfloat16 result: the 8-bit matrix instructions add 64
products after rounding each to 2^-13 of the largest one at least, so a group of
64 is off by at most 64 * 2^-13 of its largest product, on top of the above.
With a float32 result products are exact as for bf16.
"""
import numpy as np
import torch

import muon_step_03_amd as M
from oracle import linear_oracle as lin

DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def draw(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if x.numel() > 64:
        x.view(-1)[::97] *= 8.0
    return (x * scale).to(dtype).to(DEV)


def ragged(tokens, count, seed=0, before=0, behind=0):
    """Offsets of `count` matrices over the tokens between the two margins, some
    without any."""
    g = np.random.default_rng(seed)
    cuts = np.sort(g.integers(before, max(before, tokens - behind) + 1, max(0, count - 1)))
    if count > 3:
        cuts[1] = cuts[0]
    o = np.concatenate([[before], cuts, [max(before, tokens - behind)]])[:count + 1]
    return [int(v) for v in o]


def off(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int64, device=DEV)


def groups_of_largest(x, W, size=64):
    """Sum over groups of `size` along k of the largest |x| |W| product's bound:
    the product of the largest factors (at least the largest product)."""
    k = x.shape[1]
    out = np.zeros((x.shape[0], W.shape[0]))
    for i in range(0, k, size):
        out += np.abs(x[:, i:i + size]).max(1)[:, None] * np.abs(W[:, i:i + size]).max(1)[None]
    return out


def check(got, x, W, offsets, across, out_dtype, *, eight=False, exact_products=True):
    """A product against float64, elementwise."""
    got = f64(got)
    fn = lin.input_grad if across else lin.forward
    want, mag = fn(x, W, offsets), fn(np.abs(x), np.abs(W), offsets)
    k = x.shape[1]
    bound = (k + (8 if exact_products else 9)) * U * mag
    if eight and out_dtype == torch.bfloat16:
        Wn = np.swapaxes(W, -1, -2) if across else W
        if offsets is None:
            big = groups_of_largest(x, Wn)
        else:
            big, o = np.zeros(want.shape), lin.bounds(offsets, x.shape[0])
            for e in range(W.shape[0]):
                if o[e + 1] > o[e]:
                    big[o[e]:o[e + 1]] = groups_of_largest(x[o[e]:o[e + 1]], Wn[e])
        bound = bound + 64 * 2.0 ** -13 * big
        # and the errors of many elements together: far below a bf16 rounding
        off_by = np.linalg.norm(got - want)
        assert off_by <= (2.0 ** -8 + 2.0 ** -13) * np.linalg.norm(want) + 1e-300
    bound = bound + HALF[out_dtype] * (np.abs(want) + bound)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert over.size == 0 or over.max() <= 0, f"over its bound by {over.max():.3e} at {np.unravel_index(over.argmax(), over.shape)}"


def eight(x, W):
    """A checkpoint and an 8-bit weight of x and W, and their float64 values."""
    ck, w8 = M.checkpoint_save(x, "e4m3"), M.weight_quantize(W)
    xv = f64(M.checkpoint_restore(ck, torch.float32))
    Wn = f64(W)
    wv = np.stack([lin.quantized(w)[0] for w in Wn]) if Wn.ndim == 3 else lin.quantized(Wn)[0]
    return ck, w8, xv, wv
