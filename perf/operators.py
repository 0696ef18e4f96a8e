"""Cases of the 8-bit linear layer and of the LayerNorm forward.

The operators, each in a plain form made of elementary torch operations and as
the calls a user makes of the library (``own``):

    quantize   X (rows x cols) into 8-bit floats with one power-of-two scale
               per block of 128 values, along the rows, and along the columns
               (the checkpoint the backward reads), with the column sums
    forward    the activations quantised, then out = inp . weight^T + bias
               from 8-bit operands; a training call also keeps the checkpoint
    backward   dout quantised (with dbias, its column sums), then
               dinp = dout . weight and dweight (+)= dout^T . inp from 8-bit
               operands, inp being the forward's checkpoint
    layernorm  out = (inp - mean) * rstd * weight + bias, with mean and rstd
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FORMATS = {"e4m3": (torch.float8_e4m3fn, 8, 3, -6), "e5m2": (torch.float8_e5m2, 15, 2, -14)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the gradient of GPT-2 XL's MLP hidden layer, 8 x 1024 tokens: both
        # directions and the bias gradient, as a training step needs them
        dict(name="quantize-dout-xl", op="quantize", rows=8192, cols=6400, dtype="bf16", format="e5m2", sums=True),
        # an fp32 activation of ragged sizes: neither side a multiple of a block
        dict(name="quantize-ragged-f32", op="quantize", rows=1000, cols=1004, dtype="f32", format="e4m3", sums=False),
        # serving: one token through GPT-2 XL's qkv
        dict(name="forward-token", op="forward", tokens=1, C=1600, OC=4800, dtype="bf16", format="e4m3", bias=True, train=False),
        # serving: 16 sequences' next tokens through the padded GPT-2 vocabulary
        dict(name="forward-head-16", op="forward", tokens=16, C=768, OC=50304, dtype="bf16", format="e4m3", bias=False, train=False),
        # a prompt of odd length in fp32 storage, GPT-2 small's qkv
        dict(name="forward-prompt-f32", op="forward", tokens=777, C=768, OC=2304, dtype="f32", format="e4m3", bias=True, train=False),
        # training: GPT-2 XL's MLP fc, 8 x 1024 tokens, checkpoint kept
        dict(name="forward-train-xl", op="forward", tokens=8192, C=1600, OC=6400, dtype="bf16", format="e4m3", bias=True, train=True),
        # a small layer with ragged sizes everywhere
        dict(name="backward-ragged", op="backward", tokens=500, C=328, OC=520, dtype="bf16", wdtype="bf16", format="e4m3", add=False),
        # training: GPT-2 small's qkv, 8 x 1024 tokens
        dict(name="backward-small-qkv", op="backward", tokens=8192, C=768, OC=2304, dtype="bf16", wdtype="bf16", format="e4m3", add=False),
        # training: GPT-2 XL's MLP fc with an fp32 weight gradient that adds up over
        # micro-batches, dout in the wider-range format
        dict(name="backward-xl", op="backward", tokens=8192, C=1600, OC=6400, dtype="bf16", wdtype="f32", format="e5m2", add=True),
        # serving: the norm of one token
        dict(name="layernorm-token", op="layernorm", tokens=1, C=1600, dtype="bf16"),
        # training: 8 x 1024 tokens of GPT-2 XL
        dict(name="layernorm-xl", op="layernorm", tokens=8192, C=1600, dtype="bf16"),
        # fp32, an odd number of wide rows
        dict(name="layernorm-wide-f32", op="layernorm", tokens=999, C=6404, dtype="f32"),
    ]


def draw(rng):
    def size(lo, hi, step):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    dtype = rng.choice(["bf16", "f32"])
    step = 8 if dtype == "bf16" else 4
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    op = rng.choice(["quantize", "forward", "forward", "backward", "backward", "layernorm"])
    if op in ("quantize", "layernorm"):
        cols = size(8, 8192, step)
        rows = size(1, min(8192, 52_000_000 // cols), 1)
        if op == "quantize":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, format=fmt, sums=rng.random() < 0.5)
        return dict(op=op, tokens=rows, C=cols, dtype=dtype)
    C, OC = size(64, 6400, step), size(64, 12800, step)
    tokens = size(1, max(1, min(8192, 80_000_000_000 // (C * OC))), 1)
    if op == "forward":
        return dict(op=op, tokens=tokens, C=C, OC=OC, dtype=dtype, format=fmt, bias=rng.random() < 0.5,
                    train=rng.random() < 0.5)
    return dict(op=op, tokens=tokens, C=C, OC=OC, dtype=dtype, wdtype=rng.choice(["bf16", "f32"]), format=fmt,
                add=rng.random() < 0.5)


def _ld(k):
    return -(-k // 16) * 16


def _scale_bytes(rows, k):
    return -(-rows // 128) * 128 * (-(-k // (4 * BLOCK)) * 4)


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (es + 2) + 2 * (r * c // BLOCK) + (c * es if case["sums"] else 0), "flops": 0}
    t, c = case["tokens"], case["C"]
    if op == "layernorm":
        return {"bytes": 2 * t * c * es + 2 * c * es + 8 * t, "flops": 8 * t * c}
    o = case["OC"]
    if op == "forward":
        kept = t * c * 129 // 128 if case["train"] else 0
        return {"bytes": t * c * es + kept + o * c * 129 // 128 + t * o * es + (o * es if case["bias"] else 0),
                "flops": 2 * t * c * o}
    ws = 2 if case["wdtype"] == "bf16" else 4
    return {"bytes": t * o * es + t * c * 129 // 128 + o * c * 129 // 128 + t * c * es + o * es
            + o * c * ws * (2 if case["add"] else 1), "flops": 4 * t * c * o}


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activation(g, rows, cols):
    # normal values, a few channels far larger than the rest
    x = _randn(g, rows, cols)
    return x * torch.exp(0.5 * _randn(g, 1, cols)) * (1 + 12 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01))


def _gradient(g, rows, cols):
    # small values whose size differs from token to token; padding tokens have none
    x = _randn(g, rows, cols) * (0.01 * torch.exp(_randn(g, rows, 1)))
    if rows > 8:
        x[torch.rand(rows, generator=g, device="cuda") < 0.03] = 0
    return x


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    op = case["op"]
    if op == "quantize":
        make = _gradient if case["sums"] else _activation
        return {"x": make(g, case["rows"], case["cols"]).to(dt)}
    t, c = case["tokens"], case["C"]
    if op == "layernorm":
        x = _activation(g, t, c) + 0.3 * _randn(g, 1, c) + 0.1 * _randn(g, t, 1)
        return {"inp": x.to(dt), "weight": (1 + 0.2 * _randn(g, c)).to(dt), "bias": (0.1 * _randn(g, c)).to(dt)}
    o = case["OC"]
    d = {"weight": (0.02 * _randn(g, o, c)).to(dt), "inp": _activation(g, t, c).to(dt)}
    if op == "forward":
        d["bias"] = (0.1 * _randn(g, o)).to(dt) if case["bias"] else None
        return d
    d["dout"] = _gradient(g, t, o).to(dt)
    d["dweight"] = (0.1 * _randn(g, o, c)).to(TYPES[case["wdtype"]])
    return d


def _room(rows, k, fmt):
    """Buffers of an 8-bit matrix: its values and its scales."""
    return (torch.empty(rows, _ld(k), device="cuda", dtype=FORMATS[fmt][0]),
            torch.empty(_scale_bytes(rows, k), device="cuda", dtype=torch.uint8))


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        s["room"], s["room_t"] = _room(r, c, case["format"]), _room(c, r, case["format"])
        s["sums"] = torch.empty(c, device="cuda", dtype=dt) if case["sums"] else None
        return s
    t, c = case["tokens"], case["C"]
    if op == "layernorm":
        s["out"] = torch.empty(t, c, device="cuda", dtype=dt)
        s["mean"] = torch.empty(t, device="cuda")
        s["rstd"] = torch.empty(t, device="cuda")
        return s
    o = case["OC"]
    if op == "forward":
        # the weight is kept in 8 bits by the user's program
        s["w8"] = quantize(s.pop("weight").float(), case["format"])
        s["room"] = _room(t, c, case["format"])
        s["room_t"] = _room(c, t, case["format"]) if case["train"] else (None, None)
        s["out"] = torch.empty(t, o, device="cuda", dtype=dt)
        return s
    # kept from the forward: the weight's and the activation's column forms
    s["w8t"] = quantize(s.pop("weight").float().t(), "e4m3")
    s["i8t"] = quantize(s.pop("inp").float().t(), "e4m3")
    s["room"], s["room_t"] = _room(t, o, case["format"]), _room(o, t, case["format"])
    s["dinp"] = torch.empty(t, c, device="cuda", dtype=dt)
    s["dbias"] = torch.empty(o, device="cuda", dtype=dt)
    return s


# ------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in fp32 for whole e in -127 .. 127, from its bits."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def quantize(x, fmt):
    """X (rows x K, fp32) -> 8-bit values (rows x K rounded up to 16) and the
    scale bytes: the exponent (plus 127) of the smallest power of two that
    brings each block of 128 under the format's largest value, in tiles of 128
    rows x 4 blocks, row r of a tile at 16 * (r % 32) + 4 * (r // 32)."""
    f8, emax, _, _ = FORMATS[fmt]
    rows, k = x.shape
    kb = -(-k // BLOCK)
    g4, r128 = -(-kb // 4), -(-rows // 128)
    xb = torch.zeros(rows, kb * BLOCK, device=x.device)
    xb[:, :k] = x
    xb = xb.view(rows, kb, BLOCK)
    amax = torch.where(torch.isfinite(xb), xb.abs(), torch.zeros_like(xb)).amax(2)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1): the largest value is 1.75 2^emax
    s = torch.where(amax > 0, (e - 1 - emax + (m > 0.875).to(e.dtype)).clamp(min=-127), torch.zeros_like(e))
    y = xb * _pow2(-s)[:, :, None]
    y = torch.where(torch.isfinite(xb), y, torch.full_like(y, float("nan")))
    q = y.view(rows, kb * BLOCK)[:, :_ld(k)].to(f8)
    b = torch.full((r128 * 128, g4 * 4), 127, device=x.device, dtype=torch.uint8)
    b[:rows, :kb] = (s + 127).to(torch.uint8)
    return q.contiguous(), b.view(r128, 4, 32, g4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def dequantize(q8, rows, k):
    q, b = q8
    g4, r128, kb = -(-k // (4 * BLOCK)), -(-rows // 128), -(-k // BLOCK)
    e = b.view(r128, g4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r128 * 128, g4 * 4)[:rows, :kb].to(torch.int32) - 127
    return q[:, :k].float() * _pow2(e)[:, :, None].expand(rows, kb, BLOCK).reshape(rows, kb * BLOCK)[:, :k]


def _plain(s):
    case = s["case"]
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "quantize":
        x = s["x"].float()
        q, qt = quantize(x, case["format"]), quantize(x.t(), case["format"])
        return {"q": q[0], "scale": q[1], "qt": qt[0], "scale_t": qt[1],
                "sums": x.double().sum(0).to(dt) if case["sums"] else None}
    t, c = case["tokens"], case["C"]
    if op == "layernorm":
        x = s["inp"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
        return {"out": (d * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt), "mean": mean, "rstd": rstd}
    o = case["OC"]
    if op == "forward":
        x = s["inp"].float()
        i8 = quantize(x, case["format"])
        out = dequantize(i8, t, c) @ dequantize(s["w8"], o, c).t()
        if s["bias"] is not None:
            out = out + s["bias"].float()
        i8t = quantize(x.t(), case["format"]) if case["train"] else (None, None)
        return {"out": out.to(dt), "qt": i8t[0], "scale_t": i8t[1]}
    d = s["dout"].float()
    d8, d8t = quantize(d, case["format"]), quantize(d.t(), case["format"])
    dinp = (dequantize(d8, t, o) @ dequantize(s["w8t"], c, o).t()).to(dt)
    dweight = dequantize(d8t, o, t) @ dequantize(s["i8t"], c, t).t()
    if case["add"]:
        dweight = s["dweight"].float() + dweight
    s["dweight"].copy_(dweight)
    return {"dinp": dinp, "dweight": s["dweight"], "dbias": d.double().sum(0).to(dt)}


# ------------------------------------------------------------------ the library's calls

def _library(s):
    import linear_layer_gemms_gb300 as mm

    def ok(rc):
        if rc != mm.OK:
            raise mm.MmbwdError(rc)

    case = s["case"]
    op, dt = case["op"], mm.BF16 if case["dtype"] == "bf16" else mm.F32
    if op == "layernorm":
        ok(mm.lnbwd_forward(s["out"], s["mean"], s["rstd"], s["inp"], s["weight"], s["bias"], 1, case["tokens"],
                            case["C"], EPS, dt))
        return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
    fmt = mm.E4M3 if case["format"] == "e4m3" else mm.E5M2
    (q, sc), (qt, sct) = s["room"], s["room_t"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        n = mm.mmbwd_q8_quantize_workspace_bytes(r, c) if case["sums"] else 0
        ws = torch.empty(n, device="cuda", dtype=torch.uint8) if n else None
        ok(mm.mmbwd_q8_quantize(q, sc, qt, sct, s["sums"], s["x"], ws, n, r, c, dt, fmt))
        return {"q": q, "scale": sc, "qt": qt, "scale_t": sct, "sums": s["sums"]}
    t, c, o = case["tokens"], case["C"], case["OC"]
    if op == "forward":
        ok(mm.mmbwd_q8_quantize(q, sc, qt, sct, None, s["inp"], None, 0, t, c, dt, fmt))
        ok(mm.mmbwd_q8_forward(s["out"], q, sc, s["w8"][0], s["w8"][1], s["bias"], 1, t, c, o, fmt, fmt, dt))
        return {"out": s["out"], "qt": qt, "scale_t": sct}
    wdt = mm.BF16 if case["wdtype"] == "bf16" else mm.F32
    n = max(mm.mmbwd_q8_quantize_workspace_bytes(t, o), mm.mmbwd_q8_backward_workspace_bytes(1, t, c, o))
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    ok(mm.mmbwd_q8_quantize(q, sc, qt, sct, s["dbias"], s["dout"], ws, n, t, o, dt, fmt))
    ok(mm.mmbwd_q8_backward(s["dinp"], s["dweight"], q, sc, qt, sct, s["i8t"][0], s["i8t"][1], s["w8t"][0], s["w8t"][1],
                            ws, n, 1, t, c, o, fmt, mm.E4M3, mm.E4M3, dt, wdt,
                            mm.Q8_ADD_DWEIGHT if case["add"] else 0))
    return {"dinp": s["dinp"], "dweight": s["dweight"], "dbias": s["dbias"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _exact_q8(x, fmt):
    """Values, scale exponents and what they stand for, of x (rows x K, fp64)."""
    _, emax, mant, emin = FORMATS[fmt]
    rows, k = x.shape
    kb = -(-k // BLOCK)
    xb = torch.zeros(rows, kb * BLOCK, device=x.device, dtype=torch.float64)
    xb[:, :k] = x
    xb = xb.view(rows, kb, BLOCK)
    amax = xb.abs().amax(2)
    top = 1.75 * 2.0 ** emax
    s = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, top)) / top))
    s = torch.where(amax > top * torch.exp2(s), s + 1, s)  # log2 rounds: settle the borders
    s = torch.where(amax <= top * torch.exp2(s - 1), s - 1, s)
    s = torch.where(amax > 0, s.clamp(min=-127), torch.zeros_like(s))
    y = xb * torch.exp2(-s)[:, :, None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** emin))).clamp(min=emin) - mant)
    y = torch.round(y / step) * step
    z = (y * torch.exp2(s)[:, :, None]).view(rows, kb * BLOCK)[:, :k]
    return y.view(rows, kb * BLOCK)[:, :_ld(k)], s, z


def _exact_scales(s, rows, k):
    g4, r128, kb = -(-k // (4 * BLOCK)), -(-rows // 128), -(-k // BLOCK)
    at_r = torch.arange(rows, device=s.device)[:, None]
    at_k = torch.arange(kb, device=s.device)[None, :]
    flat = torch.full((_scale_bytes(rows, k),), 127, device=s.device, dtype=torch.uint8)
    flat[((at_r // 128 * g4 + at_k // 4) * 512 + at_r % 32 * 16 + at_r % 128 // 32 * 4 + at_k % 4).reshape(-1)] = \
        (s + 127).to(torch.uint8).reshape(-1)
    assert flat.numel() == r128 * g4 * 512
    return flat


def exact(case, seed):
    d = {k: v.double() if v is not None else None for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        q, s, _ = _exact_q8(d["x"], case["format"])
        qt, st, _ = _exact_q8(d["x"].t(), case["format"])
        return {"q": q, "scale": _exact_scales(s, r, c), "qt": qt, "scale_t": _exact_scales(st, c, r),
                "sums": d["x"].sum(0) if case["sums"] else None}
    t, c = case["tokens"], case["C"]
    if op == "layernorm":
        mean, var = d["inp"].mean(1), d["inp"].var(1, unbiased=False)
        rstd = torch.rsqrt(var + EPS)
        return {"out": (d["inp"] - mean[:, None]) * rstd[:, None] * d["weight"] + d["bias"], "mean": mean, "rstd": rstd}
    if op == "forward":
        out = _exact_q8(d["inp"], case["format"])[2] @ _exact_q8(d["weight"], case["format"])[2].t()
        if d["bias"] is not None:
            out = out + d["bias"]
        if not case["train"]:
            return {"out": out, "qt": None, "scale_t": None}
        qt, st, _ = _exact_q8(d["inp"].t(), case["format"])
        return {"out": out, "qt": qt, "scale_t": _exact_scales(st, c, t)}
    z = _exact_q8(d["dout"], case["format"])[2]
    dinp = z @ _exact_q8(d["weight"].t(), "e4m3")[2].t()
    dweight = _exact_q8(d["dout"].t(), case["format"])[2] @ _exact_q8(d["inp"].t(), "e4m3")[2].t()
    if case["add"]:
        dweight = dweight + d["dweight"]
    return {"dinp": dinp, "dweight": dweight, "dbias": d["dout"].sum(0)}
