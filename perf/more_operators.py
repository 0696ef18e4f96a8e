"""Cases of the block around the linear layer: the layer with an activation and a
residual in its epilogue, the norms around a block with its gate and residual
scale, and the gradients' global norm with clipping.

The operators, each in a plain form made of elementary torch operations and as
the calls a user makes of the library (``own``):

    forward        out = act(inp . weight^T + bias) + residual, pre = the
                   argument of act (kept for the backward where asked for)
    backward       of a layer whose inp is act(pre): dpre = (dout . weight) *
                   act'(pre), dweight += dout^T . inp, dbias = column sums of
                   dout; "alone" is the product with act'(pre) by itself
    norm           residual_out = x + scale * gate * post(branch) and
                   out = norm(residual_out), post and norm being a LayerNorm,
                   an RMSNorm or nothing, with the row statistics
    norm_backward  its gradients; those of the parameters add to what is there
    clip           the 2-norm over many tensors, and the tensors times
                   min(1, max_norm / (norm + 1e-6)), in other buffers or in place
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving: one token through GPT-2 XL's MLP projection, added to the residual stream
        dict(name="forward-token", op="forward", tokens=1, C=6400, OC=1600, dtype="bf16", act="none", bias=True,
             pre=False, residual=True),
        # fp32, ragged sizes everywhere, with everything the epilogue does
        dict(name="forward-ragged-f32", op="forward", tokens=333, C=772, OC=1300, dtype="f32", act="silu", bias=True,
             pre=True, residual=True),
        # training: GPT-2 XL's MLP fc, 8 x 1024 tokens, the activation's argument kept for the backward
        dict(name="forward-fc-xl", op="forward", tokens=8192, C=1600, OC=6400, dtype="bf16", act="gelu", bias=True,
             pre=True, residual=False),
        # a small layer in fp32 behind a ReLU
        dict(name="backward-ragged-f32", op="backward", alone=False, tokens=200, C=264, OC=388, dtype="f32",
             act="relu", bias=True),
        # training: GPT-2 XL's MLP projection, whose input is the GELU of the fc's output
        dict(name="backward-proj-xl", op="backward", alone=False, tokens=8192, C=6400, OC=1600, dtype="bf16",
             act="gelu", bias=True),
        # an activation that no product precedes: an odd number of tokens of GPT-2 XL's hidden layer
        dict(name="backward-alone", op="backward", alone=True, tokens=4001, C=6400, OC=0, dtype="bf16", act="gelu",
             bias=False),
        # serving: one token of GPT-2 XL, residual and the next LayerNorm
        dict(name="norm-token", op="norm", B=1, T=1, C=1600, dtype="bf16", post="none", norm="layer", gate=False,
             scale=1.0),
        # training: 8 x 1024 tokens, a norm after the block and one before the next, with a gate
        dict(name="norm-xl", op="norm", B=8, T=1024, C=1600, dtype="bf16", post="rms", norm="rms", gate=True,
             scale=0.5),
        # fp32, ragged, LayerNorms
        dict(name="norm-backward-ragged-f32", op="norm_backward", B=7, T=111, C=1004, dtype="f32", post="layer",
             norm="layer", gate=True, scale=0.7),
        # training: 8 x 1024 tokens of GPT-2 XL
        dict(name="norm-backward-xl", op="norm_backward", B=8, T=1024, C=1600, dtype="bf16", post="rms", norm="rms",
             gate=True, scale=0.5),
        # a few small tensors of odd sizes and both types, whose norm is under the limit, in place
        dict(name="clip-few", op="clip", tensors="odd", count=20, most=30011, dtype="mixed", clipped=False,
             in_place=True),
        # the gradients of GPT-2 XL's embeddings and four of its layers, clipped into the buffers that the
        # optimizer reads
        dict(name="clip-xl", op="clip", tensors="gpt2", count=4, most=1600, dtype="f32", clipped=True,
             in_place=False),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))) / step)) * step)

    op = rng.choice(["forward", "forward", "backward", "norm", "norm_backward", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 4
    if op in ("forward", "backward"):
        C, OC = size(64, 6400, step), size(64, 6400, step)
        most = 80_000_000_000 if dtype == "bf16" else 8_000_000_000
        tokens = size(1, max(1, min(8192, most // (C * OC))))
        act = rng.choice(["none", "gelu", "gelu", "silu", "relu"])
        if op == "forward":
            return dict(op=op, tokens=tokens, C=C, OC=OC, dtype=dtype, act=act, bias=rng.random() < 0.7,
                        pre=rng.random() < 0.5, residual=rng.random() < 0.5)
        return dict(op=op, alone=rng.random() < 0.2, tokens=tokens, C=C, OC=OC, dtype=dtype, act=act,
                    bias=rng.random() < 0.7)
    if op == "clip":
        return dict(op=op, tensors="odd", count=size(1, 300), most=size(1, 400_000), dtype=rng.choice(["bf16", "f32", "mixed"]),
                    clipped=True, in_place=False)
    C = size(64, 8192, step)
    rows = size(1, min(8192, 13_000_000 // C))
    B = rng.choice([1, 2, 3])
    return dict(op=op, B=B, T=max(1, rows // B), C=C, dtype=dtype, post=rng.choice(["none", "layer", "rms"]),
                norm=rng.choice(["layer", "rms"]), gate=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.144]))


def _sizes(case):
    """Values of each tensor of a clip case."""
    if case["tensors"] == "gpt2":  # token and position embeddings, then the layers' tensors, then the last norm
        c = case["most"]
        layer = [c, c, 3 * c * c, 3 * c, c * c, c, c, c, 4 * c * c, 4 * c, 4 * c * c, c]
        return [50257 * c, 1024 * c] + layer * case["count"] + [c, c]
    n, most = case["count"], case["most"]
    return [max(1, int(most ** (((i * 0.6180339887) % 1.0) ** 0.5))) for i in range(n)]


def _parts(case):
    """(type, sizes) of the tensors by type; a mixed list alternates."""
    sizes = _sizes(case)
    if case["dtype"] != "mixed":
        return [(case["dtype"], sizes)]
    return [("bf16", sizes[0::2])] + ([("f32", sizes[1::2])] if len(sizes) > 1 else [])


def work(case):
    op = case["op"]
    if op == "clip":
        moved = sum(sum(sizes) * (2 if dt == "bf16" else 4) for dt, sizes in _parts(case))
        return {"bytes": moved * (2 if case["clipped"] or not case["in_place"] else 1), "flops": 3 * sum(_sizes(case))}
    es = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_backward"):
        n, c, t = case["B"] * case["T"] * case["C"], case["C"], case["B"] * case["T"]
        stats = 4 * t * ((1 + (case["norm"] == "layer")) + (0 if case["post"] == "none" else 1 + (case["post"] == "layer")))
        cols = c * es * (_norm_params(case["norm"]) + _norm_params(case["post"]) + (1 if case["gate"] else 0))
        if op == "norm":
            return {"bytes": 4 * n * es + cols + stats, "flops": 16 * n}
        return {"bytes": 6 * n * es + 3 * cols + stats, "flops": 30 * n}
    t, c, o = case["tokens"], case["C"], case["OC"]
    if op == "forward":
        return {"bytes": es * (t * c + o * c + t * o * (1 + case["pre"] + case["residual"]) + (o if case["bias"] else 0)),
                "flops": 2 * t * c * o}
    if case["alone"]:
        return {"bytes": 3 * t * c * es, "flops": 10 * t * c}
    return {"bytes": es * (t * o + 3 * t * c + 3 * o * c + (o if case["bias"] else 0)), "flops": 4 * t * c * o}


def _norm_params(kind):
    return {"none": 0, "layer": 2, "rms": 1}[kind]


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activation(g, rows, cols):
    # normal values, a few channels larger than the rest
    x = _randn(g, rows, cols)
    return x * torch.exp(0.3 * _randn(g, 1, cols)) * (1 + 6 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01))


def _gradient(g, rows, cols):
    # small values whose size differs from token to token; padding tokens have none
    x = _randn(g, rows, cols) * (0.01 * torch.exp(0.5 * _randn(g, rows, 1)))
    if rows > 8:
        x[torch.rand(rows, generator=g, device="cuda") < 0.03] = 0
    return x


def _plain_act(x, act):
    if act == "gelu":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return torch.where(x < 0, torch.zeros_like(x), x) if act == "relu" else x


def _plain_slope(x, act):
    if act == "gelu":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    return (x > 0).to(x.dtype) if act == "relu" else torch.ones_like(x)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "clip":
        d = {}
        for dt, sizes in _parts(case):
            # one buffer of a type, each tensor at a multiple of eight values, as an arena holds them
            starts, at = [], 0
            for n in sizes:
                starts.append(at)
                at += -(-n // 8) * 8
            flat = (_randn(g, at) * 0.003).to(TYPES[dt])
            inside = torch.zeros(at + 1, device="cuda", dtype=torch.int32)
            inside[torch.tensor(starts, device="cuda")] += 1
            inside.index_add_(0, torch.tensor([a + n for a, n in zip(starts, sizes)], device="cuda"),
                              torch.full((len(sizes),), -1, device="cuda", dtype=torch.int32))
            flat *= (torch.cumsum(inside, 0)[:at] > 0).to(flat.dtype)
            d[dt] = flat
            d[dt + "_at"] = list(zip(starts, sizes))
        return d
    dt = TYPES[case["dtype"]]
    if op in ("norm", "norm_backward"):
        t, c = case["B"] * case["T"], case["C"]
        d = {"x": _activation(g, t, c) + 0.3 * _randn(g, 1, c), "branch": 0.5 * _activation(g, t, c) + 0.1 * _randn(g, 1, c)}
        d["gate"] = 0.5 + 0.3 * _randn(g, c) if case["gate"] else None
        for k, kind in (("_post", case["post"]), ("", case["norm"])):
            d["weight" + k] = 1 + 0.2 * _randn(g, c) if kind != "none" else None
            d["bias" + k] = 0.1 * _randn(g, c) if kind == "layer" else None
        if op == "norm_backward":
            d["residual"] = d.pop("x")
            d["dout"], d["dresidual"] = _gradient(g, t, c), _gradient(g, t, c)
            for k in ("gate", "weight_post", "bias_post", "weight", "bias"):
                d["d" + k] = 0.1 * _randn(g, c) if d[k] is not None else None
            d.pop("bias")  # the gradients do not need it
        return {k: v if v is None else v.to(dt) for k, v in d.items()}
    t, c, o = case["tokens"], case["C"], case["OC"]
    if op == "forward":
        d = {"inp": _activation(g, t, c), "weight": 0.7 / math.sqrt(c) * _randn(g, o, c),
             "bias": 0.1 * _randn(g, o) if case["bias"] else None,
             "residual": _activation(g, t, o) if case["residual"] else None}
    elif case["alone"]:
        d = {"pre": _activation(g, t, c), "dout": _gradient(g, t, c)}
    else:
        d = {"pre": _activation(g, t, c), "dout": _gradient(g, t, o), "weight": 0.02 * _randn(g, o, c),
             "dweight": 0.05 * _randn(g, o, c)}
    d = {k: v if v is None else v.to(dt) for k, v in d.items()}
    if op == "backward" and not case["alone"]:
        d["inp"] = _plain_act(d["pre"].float(), case["act"]).to(dt)  # what the forward kept
    return d


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    op = case["op"]
    if op == "clip":
        s["norm"] = torch.empty(1, device="cuda")
        total, pairs = torch.zeros((), device="cuda", dtype=torch.float64), []
        for dt, _ in _parts(case):
            flat = s[dt]
            s[dt + "_out"] = flat if case["in_place"] else torch.zeros_like(flat)
            pairs += [(flat[a:a + n], s[dt + "_out"][a:a + n], n, dt) for a, n in s[dt + "_at"]]
            total += sum((x.double().square().sum() for x in flat.split(1 << 26)), torch.zeros_like(total))
        s["pairs"] = pairs
        s["max_norm"] = float(total.sqrt()) * (0.37 if case["clipped"] else 1.5)
        return s
    dt = TYPES[case["dtype"]]
    if op in ("norm", "norm_backward"):
        t, c = case["B"] * case["T"], case["C"]
        rows = lambda: torch.empty(t, c, device="cuda", dtype=dt)  # noqa: E731
        if op == "norm":
            s["out"], s["residual_out"] = rows(), rows()
            for k, kind in (("_post", case["post"]), ("", case["norm"])):
                s["mean" + k] = torch.empty(t, device="cuda") if kind == "layer" else None
                s["rstd" + k] = torch.empty(t, device="cuda") if kind != "none" else None
            return s
        s["dx"], s["dbranch"] = rows(), rows()
        for k, kind, of in (("_post", case["post"], s["branch"]), ("", case["norm"], s["residual"])):
            # kept by the forward
            v = of.double()
            mean = v.mean(1) if kind == "layer" else None
            v = v if mean is None else v - mean[:, None]
            s["mean" + k] = None if mean is None else mean.float()
            s["rstd" + k] = (1 / (v.square().mean(1) + EPS).sqrt()).float() if kind != "none" else None
        return s
    t, c, o = case["tokens"], case["C"], case["OC"]
    if op == "forward":
        s["out"] = torch.empty(t, o, device="cuda", dtype=dt)
        s["pre"] = torch.empty(t, o, device="cuda", dtype=dt) if case["pre"] else None
        return s
    s["dpre"] = torch.empty(t, c, device="cuda", dtype=dt)
    if not case["alone"]:
        s["dbias"] = torch.empty(o, device="cuda", dtype=dt) if case["bias"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_norm(v, kind, weight, bias):
    """(normalised rows, the result, mean, rstd) in 32 bits."""
    if kind == "none":
        return v, v, None, None
    mean = v.mean(1) if kind == "layer" else None
    d = v if mean is None else v - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    n = d * rstd[:, None]
    y = n * weight.float()
    return n, y if bias is None else y + bias.float(), mean, rstd


def _plain_norm_gradient(g, n, rstd, kind):
    """Through the normalisation, from the gradient `g` of the normalised rows."""
    if kind == "none":
        return g
    d = g - n * (g * n).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d * rstd[:, None]


def _plain_normalised(v, kind, mean, rstd):
    if kind == "none":
        return v
    return (v if mean is None else v - mean[:, None]) * rstd[:, None]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), device="cuda", dtype=torch.float64)
        for dt, _ in _parts(case):
            total = total + sum(x.double().square().sum() for x in s[dt].split(1 << 26))
        norm = total.sqrt().float().reshape(1)
        coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        for dt, _ in _parts(case):
            s[dt + "_out"].copy_(s[dt].float() * coef)
        return {"norm": norm, **{dt: s[dt + "_out"] for dt, _ in _parts(case)}}
    dt = TYPES[case["dtype"]]
    f = {k: v.float() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if op == "norm":
        z, y, mean_post, rstd_post = _plain_norm(f["branch"], case["post"], s["weight_post"], s["bias_post"])
        r = f["x"] + case["scale"] * (y if s["gate"] is None else y * f["gate"])
        _, out, mean, rstd = _plain_norm(r, case["norm"], s["weight"], s["bias"])
        return {"out": out.to(dt), "residual_out": r.to(dt), "mean_post": mean_post, "rstd_post": rstd_post,
                "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        n = _plain_normalised(f["residual"], case["norm"], s["mean"], s["rstd"])
        dr = f["dresidual"] + _plain_norm_gradient(f["dout"] * f["weight"], n, s["rstd"], case["norm"])
        z = _plain_normalised(f["branch"], case["post"], s["mean_post"], s["rstd_post"])
        y = z if case["post"] == "none" else z * f["weight_post"] + (0 if s["bias_post"] is None else f["bias_post"])
        dy = case["scale"] * (dr if s["gate"] is None else dr * f["gate"])
        g = dy if case["post"] == "none" else dy * f["weight_post"]
        out = {"dx": dr.to(dt), "dbranch": _plain_norm_gradient(g, z, s["rstd_post"], case["post"]).to(dt)}
        sums = {"dgate": case["scale"] * dr * y, "dweight_post": dy * z, "dbias_post": dy, "dweight": f["dout"] * n,
                "dbias": f["dout"]}
        for k, v in sums.items():
            if s[k] is not None:
                s[k].copy_(f[k] + v.double().sum(0))
                out[k] = s[k]
        return out
    if op == "forward":
        pre = f["inp"] @ f["weight"].t()
        if s["bias"] is not None:
            pre = pre + f["bias"]
        out = _plain_act(pre, case["act"])
        if s["residual"] is not None:
            out = out + f["residual"]
        return {"out": out.to(dt), "pre": pre.to(dt) if case["pre"] else None}
    if case["alone"]:
        return {"dpre": (f["dout"] * _plain_slope(f["pre"], case["act"])).to(dt)}
    dpre = (f["dout"] @ f["weight"]) * _plain_slope(f["pre"], case["act"])
    s["dweight"].copy_(f["dweight"] + f["dout"].t() @ f["inp"])
    return {"dpre": dpre.to(dt), "dweight": s["dweight"],
            "dbias": s["dout"].double().sum(0).to(dt) if case["bias"] else None}


# ------------------------------------------------------------------ the library's calls

def _library(s):
    import linear_layer_gemms_gb300 as mm

    def ok(rc):
        if rc != mm.OK:
            raise mm.MmbwdError(rc)

    def room(n):  # kept by the program from call to call
        if "workspace" not in s:
            s["workspace"] = torch.empty(max(n(), 1), device="cuda", dtype=torch.uint8)
        return s["workspace"], s["workspace"].numel()

    case = s["case"]
    op = case["op"]
    kinds = {"bf16": mm.BF16, "f32": mm.F32}
    if op == "clip":
        if "list" not in s:
            s["list"] = mm.grad_list([(g, None if case["in_place"] else o, n, kinds[dt]) for g, o, n, dt in s["pairs"]])
        ws, n = room(lambda: mm.mmbwd_grad_workspace_bytes(s["list"]))
        ok(mm.mmbwd_grad_clip(s["norm"], s["list"], s["max_norm"], ws, n))
        return {"norm": s["norm"], **{dt: s[dt + "_out"] for dt, _ in _parts(case)}}
    dt = kinds[case["dtype"]]
    if op in ("norm", "norm_backward"):
        names = {"none": mm.NORM_NONE, "layer": mm.NORM_LAYER, "rms": mm.NORM_RMS}
        post, norm = names[case["post"]], names[case["norm"]]
        B, T, C = case["B"], case["T"], case["C"]
        if op == "norm":
            ok(mm.lnbwd_residual_forward(s["out"], s["residual_out"], s["mean_post"], s["rstd_post"], s["mean"], s["rstd"],
                                  s["x"], s["branch"], s["gate"], s["weight_post"], s["bias_post"], s["weight"],
                                  s["bias"], B, T, C, case["scale"], EPS, post, norm, dt))
            return {k: s[k] for k in ("out", "residual_out", "mean_post", "rstd_post", "mean", "rstd")}
        ws, n = room(lambda: mm.lnbwd_residual_backward_workspace_bytes(B, T, C, dt))
        ok(mm.lnbwd_residual_backward(s["dx"], s["dbranch"], s["dgate"], s["dweight_post"], s["dbias_post"], s["dweight"],
                               s["dbias"], s["dout"], s["dresidual"], s["residual"], s["branch"], s["gate"],
                               s["weight_post"], s["bias_post"], s["weight"], s["mean_post"], s["rstd_post"], s["mean"],
                               s["rstd"], ws, n, B, T, C, case["scale"], post, norm, dt))
        out = {k: s[k] for k in ("dx", "dbranch", "dgate", "dweight_post", "dbias_post", "dweight", "dbias")}
        return {k: v for k, v in out.items() if v is not None}
    acts = {"none": mm.ACT_NONE, "gelu": mm.ACT_GELU, "silu": mm.ACT_SILU, "relu": mm.ACT_RELU}
    act, t, c, o = acts[case["act"]], case["tokens"], case["C"], case["OC"]
    if op == "forward":
        ok(mm.mmbwd_forward_act(s["out"], s["pre"], s["inp"], s["weight"], s["bias"], s["residual"], 1, t, c, o, act, dt))
        return {"out": s["out"], "pre": s["pre"]}
    if case["alone"]:
        ok(mm.mmbwd_act_backward(s["dpre"], s["dout"], s["pre"], t * c, act, dt))
        return {"dpre": s["dpre"]}
    ws, n = room(lambda: mm.mmbwd_run_act_workspace_bytes(1, t, c, o, dt))
    ok(mm.mmbwd_run_act(s["dpre"], s["dweight"], s["dbias"], s["dout"], s["inp"], s["weight"], s["pre"], ws, n, 1, t, c,
                        o, act, dt))
    return {"dpre": s["dpre"], "dweight": s["dweight"], "dbias": s["dbias"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _exact_act(x, act):
    if act == "gelu":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    if act == "silu":
        return x * torch.sigmoid(x)
    return torch.relu(x) if act == "relu" else x * 1


def _exact_norm(v, kind, weight, bias):
    if kind == "none":
        return v, None, None
    mean, var = (v.mean(1), v.var(1, unbiased=False)) if kind == "layer" else (torch.zeros_like(v[:, 0]), (v ** 2).mean(1))
    rstd = torch.rsqrt(var + EPS)
    y = (v - mean[:, None]) * rstd[:, None] * weight
    return y if bias is None else y + bias, mean if kind == "layer" else None, rstd


def exact(case, seed):
    op = case["op"]
    if op == "clip":
        d = _inputs(case, seed)
        kinds = [dt for dt, _ in _parts(case)]
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(d[dt], dtype=torch.float64)) ** 2 for dt in kinds))
        coef = min(1.0, norm * (0.37 if case["clipped"] else 1.5) / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64), **{dt: d[dt].double() * coef for dt in kinds}}
    d = {k: v.double() if v is not None else None for k, v in _inputs(case, seed).items()}
    if op == "norm":
        y, mean_post, rstd_post = _exact_norm(d["branch"], case["post"], d["weight_post"], d["bias_post"])
        r = d["x"] + case["scale"] * (1 if d["gate"] is None else d["gate"]) * y
        out, mean, rstd = _exact_norm(r, case["norm"], d["weight"], d["bias"])
        return {"out": out, "residual_out": r, "mean_post": mean_post, "rstd_post": rstd_post, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        # from the definition, by differentiating it
        with torch.enable_grad():
            old = {k: d.pop(k) for k in ("dgate", "dweight_post", "dbias_post", "dweight", "dbias")}
            v = {k: d[k].requires_grad_() for k in ("residual", "branch", "gate", "weight_post", "bias_post", "weight")
                 if d[k] is not None}
            zero = torch.zeros_like(v["weight"]).requires_grad_() if old["dbias"] is not None else None
            out, _, _ = _exact_norm(v["residual"], case["norm"], v["weight"], zero)
            first = [v["residual"], v["weight"]] + ([zero] if zero is not None else [])
            got = torch.autograd.grad((out * d["dout"]).sum() + (v["residual"] * d["dresidual"]).sum(), first)
            dr, sums = got[0], {"dweight": got[1], "dbias": got[2] if zero is not None else None}
            y, _, _ = _exact_norm(v["branch"], case["post"], v.get("weight_post"), v.get("bias_post"))
            z = case["scale"] * (v["gate"] * y if "gate" in v else y)
            names = [k for k in ("branch", "gate", "weight_post", "bias_post") if k in v]
            sums.update({"d" + k: x for k, x in zip(names, torch.autograd.grad((z * dr).sum(), [v[k] for k in names]))})
        res = {"dx": dr, "dbranch": sums.pop("dbranch")}
        res.update({k: old[k] + x for k, x in sums.items() if x is not None})
        return {k: x.detach() for k, x in res.items()}
    if op == "forward":
        pre = torch.einsum("tc,oc->to", d["inp"], d["weight"]) + (0 if d["bias"] is None else d["bias"])
        out = _exact_act(pre, case["act"]) + (0 if d["residual"] is None else d["residual"])
        return {"out": out, "pre": pre if case["pre"] else None}
    with torch.enable_grad():
        p = d["pre"].requires_grad_()
        h = _exact_act(p, case["act"])
        dh = d["dout"] if case["alone"] else torch.einsum("to,oc->tc", d["dout"], d["weight"])
        (dpre,) = torch.autograd.grad(h, p, dh)
    if case["alone"]:
        return {"dpre": dpre}
    return {"dpre": dpre, "dweight": d["dweight"] + torch.einsum("to,tc->oc", d["dout"], d["inp"]),
            "dbias": d["dout"].sum(0) if case["bias"] else None}
