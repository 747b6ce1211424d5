"""What is measured of the layer operators: layer norm's two passes, activation
checkpoints in 8 bits, and the weight gradient that reads such a checkpoint.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, where ``own`` is true, makes the
calls that a training program makes of ``muon_step_03_amd``.

Sizes are those of the hidden weights that the Muon step updates: GPT-160M and
GPT-400M (hidden 768 and 1024, MLP 4096), the MoE (hidden 512, experts of
1408, 64 routed and one shared), the 2k-hidden model (5632), and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32          # columns that share one scale of a checkpoint
E_MIN = -117        # smallest scale exponent: every value of a checkpoint is a normal number
FORMATS = {  # storage, largest magnitude, its binary exponent (value = m 2^k, m in [0.5, 1)) and m, largest scale exponent
    "e4m3": (torch.float8_e4m3fn, 448.0, 9, 0.875, 119),
    "int8": (torch.int8, 127.0, 7, 127.0 / 128.0, 121),
}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# The largest work that a listed case asks for, which bounds the drawn ones.
MOST_ELEMENTS = 1 << 27
MOST_FLOPS = 2 * 16384 * 1024 * 4096


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a layer's input norm in training on GPT-400M: 8 sequences of 2048
        # tokens; y goes on in bf16 and is kept in 8 bits for the weight gradient
        dict(name="forward gpt400m", op="forward", tokens=16384, cols=1024, dtype="bf16",
             pdtype="bf16", bias=True, fmt="e4m3"),
        # the same on one short sequence of GPT-160M, nothing kept: latency
        dict(name="forward short", op="forward", tokens=12, cols=768, dtype="bf16",
             pdtype="f32", bias=True, fmt="none"),
        # float32 training, an odd width and batch
        dict(name="forward odd f32", op="forward", tokens=4099, cols=1411, dtype="f32",
             pdtype="f32", bias=False, fmt="int8"),
        # its backward pass on GPT-400M, the input kept in 8 bits
        dict(name="backward gpt400m", op="backward", tokens=16384, cols=1024, dtype="bf16",
             pdtype="bf16", bias=True, fmt="e4m3"),
        # a short sequence of GPT-160M, the input kept as it was: latency
        dict(name="backward short", op="backward", tokens=64, cols=768, dtype="bf16",
             pdtype="f32", bias=True, fmt="none"),
        # float32 training, an odd width and batch
        dict(name="backward odd f32", op="backward", tokens=4099, cols=1411, dtype="f32",
             pdtype="f32", bias=False, fmt="none"),
        # the widest activation of a layer (the MLP's hidden one), kept and brought back
        dict(name="checkpoint wide", op="checkpoint", tokens=32768, cols=4096, dtype="bf16",
             fmt="e4m3"),
        # a small odd one in float32
        dict(name="checkpoint odd f32", op="checkpoint", tokens=501, cols=777, dtype="f32",
             fmt="int8"),
        # the MLP-up gradient of GPT-400M over 8 sequences of 2048 tokens
        dict(name="weight gpt400m up", op="weight", tokens=16384, cols=1024, rows=4096, experts=0,
             dtype="bf16", gdtype="bf16", fmt="e4m3", accumulate=False),
        # the up projections of one MoE layer's experts: ragged groups, some without a token
        dict(name="weight moe experts", op="weight", tokens=49152, cols=512, rows=1408, experts=64,
             dtype="bf16", gdtype="bf16", fmt="int8", accumulate=False),
        # a short micro-batch added to a float32 gradient of an attention projection
        dict(name="weight short", op="weight", tokens=96, cols=768, rows=768, experts=0,
             dtype="bf16", gdtype="f32", fmt="e4m3", accumulate=True),
        # float32 training, odd sizes
        dict(name="weight odd f32", op="weight", tokens=2049, cols=777, rows=1001, experts=0,
             dtype="f32", gdtype="f32", fmt="int8", accumulate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A width: any number, or one of the multiples of 64 that models have."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["forward", "backward", "checkpoint", "weight", "weight"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    fmt = rng.choice(["e4m3", "int8"])
    if op != "weight":
        cols = _size(rng, 48, 5632)
        tokens = _log(rng, 1, min(32768, MOST_ELEMENTS // cols))
        case = dict(op=op, tokens=tokens, cols=cols, dtype=dtype, fmt=fmt)
        if op != "checkpoint":
            case["fmt"] = rng.choice([fmt, fmt, "none"])
            case["pdtype"] = rng.choice([dtype, "f32"])
            case["bias"] = rng.random() < 0.7
        return case
    experts = rng.choice([0, 0, rng.randint(2, 64)])
    rows, cols = _size(rng, 64, 4096), _size(rng, 64, 4096)
    while max(1, experts) * rows * cols > 64 * 512 * 1408:
        rows, cols = max(64, rows // 2), max(64, cols // 2)
    tokens = _log(rng, 16, min(49152, MOST_FLOPS // (2 * rows * cols)))
    return dict(op=op, tokens=tokens, cols=cols, rows=rows, experts=experts, dtype=dtype,
                gdtype=rng.choice([dtype, "f32"]), fmt=fmt, accumulate=rng.random() < 0.3)


# ----------------------------------------------------------------- the inputs
def _hidden(gen, tokens, cols, dtype, dev):
    """Hidden states: unit normal tokens of differing size, a few large channels."""
    x = torch.randn(tokens, cols, generator=gen, device=dev)
    x *= torch.exp(0.3 * torch.randn(tokens, 1, generator=gen, device=dev))
    x *= 1.0 + 9.0 * (torch.rand(cols, generator=gen, device=dev) < 0.01)
    x += 0.1 * torch.randn(cols, generator=gen, device=dev)
    return x.to(dtype)


def _grad(gen, tokens, cols, dtype, dev):
    g = torch.randn(tokens, cols, generator=gen, device=dev)
    g *= 1e-3 * torch.exp(0.5 * torch.randn(tokens, 1, generator=gen, device=dev))
    return g.to(dtype)


def _offsets(seed, tokens, experts):
    """Tokens of each expert under an uneven router (about one expert in
    sixteen gets none), as their running total."""
    gen = torch.Generator().manual_seed(seed)
    p = torch.exp(0.7 * torch.randn(experts, generator=gen))
    p[torch.rand(experts, generator=gen) < 1 / 16] = 0.0
    if float(p.sum()) == 0.0:
        p[0] = 1.0
    picks = torch.multinomial(p, tokens, replacement=True, generator=gen)
    counts = torch.bincount(picks, minlength=experts)
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]), int(counts.max())


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    op, tokens, cols = case["op"], case["tokens"], case["cols"]
    dtype = DTYPES[case["dtype"]]
    x = _hidden(gen, tokens, cols, dtype, dev)
    if op in ("forward", "backward"):
        pdtype = DTYPES[case["pdtype"]]
        s["gain"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device=dev)).to(pdtype)
        s["b"] = (0.1 * torch.randn(cols, generator=gen, device=dev)).to(pdtype) if case["bias"] else None
    if op in ("forward", "checkpoint"):
        s["x"] = x
    if op == "backward":
        wide = x.double()
        mean = wide.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = torch.rsqrt((wide - mean[:, None]).square().mean(1) + EPS).float()
        s["dy"] = _grad(gen, tokens, cols, dtype, dev)
        s["x"] = x if case["fmt"] == "none" else None
    if op == "weight" or (op == "backward" and case["fmt"] != "none"):
        # what the forward pass kept: 8-bit values and the exponents of their blocks
        s["q"], s["scale"] = _quantise(x, case["fmt"])
    if op == "weight":
        s["dy"] = _grad(gen, tokens, case["rows"], dtype, dev)
        s["offsets"], s["longest"] = None, tokens
        if case["experts"]:
            offsets, s["longest"] = _offsets(seed, tokens, case["experts"])
            s["offsets"] = offsets.to(dev)
        if case["accumulate"]:
            shape = ([case["experts"]] if case["experts"] else []) + [case["rows"], cols]
            s["G"] = (1e-3 * torch.randn(shape, generator=gen, device=dev)).to(DTYPES[case["gdtype"]])
    return s


# ------------------------------------------------------------ the plain forms
def _quantise(x, fmt):
    """(q, scale) of a checkpoint: q [tokens, columns up to a multiple of 32]
    in 8 bits, scale [tokens, blocks up to a multiple of 4] in bytes e + 127.
    A block of 32 columns shares 2^e, the smallest power of two that brings
    its largest magnitude into the format's range (255 marks a block that
    holds an infinity or a NaN)."""
    store, top, k_top, m_top, e_max = FORMATS[fmt]
    tokens, cols = x.shape
    blocks = -(-cols // BLOCK)
    pad = torch.zeros(tokens, blocks * BLOCK, device=x.device)
    pad[:, :cols] = x
    pad = pad.view(tokens, blocks, BLOCK)
    large = pad.abs().amax(2)
    fine = torch.isfinite(large)
    m, k = torch.frexp(torch.where(fine, large, 0.0))
    e = (k - k_top + (m > m_top)).clamp(E_MIN, e_max)
    e = torch.where(large > 0, e, E_MIN)
    v = (pad * _power(-e)[:, :, None]).clamp(-top, top)
    v = torch.where(fine[:, :, None], v, 0.0)
    q = (v if store.is_floating_point else v.round()).to(store).view(tokens, blocks * BLOCK)
    scale = torch.zeros(tokens, _up(blocks, 4), dtype=torch.uint8, device=x.device)
    scale[:, :blocks] = torch.where(fine, e + 127, 255).to(torch.uint8)
    return q, scale


def _power(e):
    """2^e in float32, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _values(q, scale, cols):
    """The float32 values that a checkpoint stands for."""
    tokens, wide = q.shape
    blocks = wide // BLOCK
    b = scale[:, :blocks].to(torch.int32)
    p = torch.where(b == 255, float("nan"), _power(b - 127))
    return (q.float().view(tokens, blocks, BLOCK) * p[:, :, None]).view(tokens, wide)[:, :cols]


def _forward(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None] * s["gain"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = y.to(s["x"].dtype)
    out = dict(y=y, mean=mean, rstd=rstd)
    if s["fmt"] != "none":
        out["kept"] = _values(*_quantise(y, s["fmt"]), s["cols"]).to(torch.bfloat16)
    return out


def _backward(s):
    x = s["x"].float() if s["fmt"] == "none" else _values(s["q"], s["scale"], s["cols"])
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    gdy = dy * s["gain"].float()
    dx = (gdy - gdy.mean(1, keepdim=True) - xhat * (gdy * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    out = dict(dx=dx.to(s["dy"].dtype), dgain=(dy * xhat).sum(0).to(s["gain"].dtype))
    if s["b"] is not None:
        out["dbias"] = dy.sum(0).to(s["b"].dtype)
    return out


def _weight(s):
    x, dy = _values(s["q"], s["scale"], s["cols"]), s["dy"].float()
    if s["offsets"] is None:
        g = dy.t() @ x
    else:
        # each expert's tokens, laid out to the longest one's length
        begin, end = s["offsets"][:-1, None], s["offsets"][1:, None]
        at = begin + torch.arange(s["longest"], device=dy.device)
        live = (at < end)[:, :, None]
        at = at.clamp(max=dy.shape[0] - 1)
        g = torch.where(live, dy[at], 0.0).transpose(1, 2) @ torch.where(live, x[at], 0.0)
    if s["accumulate"]:
        return s["G"].copy_(s["G"].float() + g)
    return g.to(DTYPES[s["gdtype"]])


# ------------------------------------------------------ the framework's calls
def _own(s):
    import muon_step_03_amd as M
    op = s["op"]
    if op == "forward":
        r = M.layernorm_forward(s["x"], s["gain"], s["b"], eps=EPS,
                                y_checkpoint=None if s["fmt"] == "none" else s["fmt"])
        out = dict(y=r.y, mean=r.mean, rstd=r.rstd)
        if s["fmt"] != "none":
            out["kept"] = M.checkpoint_restore(r.y_checkpoint, torch.bfloat16)
        return out
    if op == "checkpoint":
        return M.checkpoint_restore(M.checkpoint_save(s["x"], s["fmt"]), torch.bfloat16)
    kept = s["x"] if s.get("x") is not None else M.ActCheckpoint(s["q"], s["scale"], s["cols"])
    if op == "backward":
        dx, dgain, dbias = M.layernorm_backward(s["dy"], kept, s["gain"], s["mean"], s["rstd"],
                                                bias=s["b"] is not None)
        out = dict(dx=dx, dgain=dgain)
        if dbias is not None:
            out["dbias"] = dbias
        return out
    return M.weight_grad(s["dy"], kept, offsets=s["offsets"], G=s.get("G"),
                         dtype=DTYPES[s["gdtype"]], accumulate=s["accumulate"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "checkpoint":
        return _values(*_quantise(state["x"], state["fmt"]), state["cols"]).to(torch.bfloat16)
    return {"forward": _forward, "backward": _backward, "weight": _weight}[op](state)


# ---------------------------------------------------------- what they have to do
def work(case):
    op, t, c = case["op"], case["tokens"], case["cols"]
    es = 2 if case["dtype"] == "bf16" else 4
    kept = t * c * (1 + 1 / BLOCK)   # a checkpoint's bytes
    if op == "checkpoint":
        return {"bytes": t * c * es + 2 * kept + 2 * t * c, "flops": 0}
    if op == "weight":
        g = max(1, case["experts"]) * case["rows"] * c * (2 if case["gdtype"] == "bf16" else 4)
        return {"bytes": t * case["rows"] * es + kept + g * (2 if case["accumulate"] else 1),
                "flops": 2 * t * case["rows"] * c}
    ps = (2 if case["pdtype"] == "bf16" else 4) * c * (2 if case["bias"] else 1)
    if op == "forward":
        more = 0 if case["fmt"] == "none" else 2 * kept + 2 * t * c
        return {"bytes": 2 * t * c * es + 8 * t + ps + more, "flops": 8 * t * c}
    read = kept if case["fmt"] != "none" else t * c * es
    return {"bytes": 2 * t * c * es + read + 8 * t + ps + c * (2 if case["pdtype"] == "bf16" else 4),
            "flops": 14 * t * c}


# ------------------------------------------------ the definition, in 64 bits
def _nearest(v, fmt):
    """Round half to even onto the format's numbers (|v| within its range)."""
    if fmt == "int8":
        return torch.round(v)
    size = torch.frexp(v).exponent.double() - 1          # floor(log2 |v|)
    step = torch.exp2(torch.clamp(size, min=-6.0) - 3)   # 3 bits behind the leading one
    return torch.round(v / step) * step


def _kept64(x, fmt):
    """What a checkpoint of x (float64) brings back."""
    top = FORMATS[fmt][1]
    out = torch.empty_like(x)
    n = x.shape[1]
    whole = n // BLOCK * BLOCK
    for part, lo, hi in ((BLOCK, 0, whole), (n - whole, whole, n)):
        if hi == lo:
            continue
        b = x[:, lo:hi].reshape(x.shape[0], -1, part)
        a = b.abs().amax(2, keepdim=True)
        e = torch.frexp(a / top).exponent.double()       # 2^(e-1) <= a / top < 2^e
        e = torch.where(a / top == torch.exp2(e - 1), e - 1, e)
        e = torch.where(a > 0, e.clamp(-117, FORMATS[fmt][4]), -117.0)
        v = (b / torch.exp2(e)).clamp(-top, top)
        out[:, lo:hi] = (_nearest(v, fmt) * torch.exp2(e)).reshape(x.shape[0], hi - lo)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    if op == "checkpoint":
        return _kept64(s["x"].double(), case["fmt"])
    if op == "forward":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * s["gain"].double()
        if s["b"] is not None:
            y += s["b"].double()
        out = dict(y=y, mean=mean, rstd=1 / torch.sqrt(var + EPS))
        if case["fmt"] != "none":
            out["kept"] = _kept64(y.to(s["x"].dtype).double(), case["fmt"])
        return out
    if "q" in s:
        e = s["scale"].double().repeat_interleave(BLOCK, 1)[:, :cols] - 127
        x = s["q"].double()[:, :cols] * torch.exp2(e)
    else:
        x = s["x"].double()
    dy = s["dy"].double()
    if op == "backward":
        r = s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * r
        a = dy * s["gain"].double()
        # the Jacobian of the normalisation applied to a, row by row
        along = (a * xhat).sum(1, keepdim=True) / cols
        out = dict(dx=r * (a - a.sum(1, keepdim=True) / cols - along * xhat),
                   dgain=torch.einsum("tc,tc->c", dy, xhat))
        if s["b"] is not None:
            out["dbias"] = dy.sum(0)
        return out
    ends = [0, case["tokens"]] if s["offsets"] is None else s["offsets"].tolist()
    g = torch.stack([dy[a:b].t() @ x[a:b] for a, b in zip(ends[:-1], ends[1:])])
    if s["offsets"] is None:
        g = g[0]
    return g + s["G"].double() if case["accumulate"] else g
