"""The operators around the linear layer in 64 bits, from their definitions, with
bounds of what 32-bit arithmetic may lose: each function takes and returns float64
tensors, on whatever device they are."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24  # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the stored type (2^-8 for bf16), relative
TINY = {"bf16": 2.0 ** -133, "f32": 2.0 ** -148}  # one step at zero
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "gelu", "silu", "relu"]
KINDS = ["none", "layer", "rms"]
EPS = 1e-5


def rounded(x, dtype):
    """x as it is stored, back in 64 bits."""
    return x.to(TDT[dtype]).double()


def normal(seed, *shape, std=1.0, device="cuda"):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(device)


def stored(err, ref, dtype):
    """`err` with the rounding of `ref` to its type."""
    return err + HALF[dtype] * (ref.abs() + err) + TINY[dtype]


def check(got, want, bound, what=""):
    """|got - want| <= bound, NaN where NaN, the same infinities."""
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(torch.where(inf, want, 0.0 * want.nan_to_num(0, 0, 0)),
                       torch.where(inf, g, 0.0 * g.nan_to_num(0, 0, 0))), f"{what}: infinities differ"
    ok = ~(nan | inf)
    over = ((g - want).abs() - bound)[ok]
    if over.numel():
        worst = over.max().item()
        assert worst <= 0, f"{what}: {worst:.3g} over the bound, {(over > 0).sum().item()} of {over.numel()}"


# ------------------------------------------------------------------ activations

def logistic_argument(x, act):
    """v with act(x) = x * sigma(v)."""
    return 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3) if act == "gelu" else x


def act_value(x, act):
    if act in ("gelu", "silu"):
        return x * torch.sigmoid(logistic_argument(x, act))
    return torch.where(x < 0, torch.zeros_like(x), x) if act == "relu" else x.clone()


def act_slope(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return torch.where(torch.isnan(x), x, (x > 0).double())
    far = x.clamp(-1e3, 1e3)  # the limits at the infinities
    v = logistic_argument(far, act)
    dv = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * far ** 2) if act == "gelu" else torch.ones_like(far)
    s = torch.sigmoid(v)
    return s + torch.where(v.abs() > 700, 0 * far, far * s * torch.sigmoid(-v) * dv)


def act_value_bound(x, act):
    """What fp32 loses in act(x): v is off by 4 steps of itself and the exponential by
    2 + 1.2 |v| of its own (the documented bound of __expf, which is above expf's), so the
    logistic function by as much, relatively, and the quotient by two more. Beyond
    |v| = 87 the exponential may leave fp32's range: the value is then below 2^-120 |x|."""
    if act in ("none", "relu"):
        return 0 * x
    v = logistic_argument(x, act).abs().clamp(max=100)
    return act_value(x, act).abs().nan_to_num(0) * (10 + 6 * v) * 2 * U + x.abs().nan_to_num(0, 0, 0) * 2.0 ** -120


def act_slope_bound(x, act):
    """Likewise of act'(x) = sigma + x sigma (1 - sigma) v'."""
    if act in ("none", "relu"):
        return 0 * x
    far = x.nan_to_num(0).clamp(-20, 20)
    v = logistic_argument(far, act)
    dv = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * far ** 2) if act == "gelu" else torch.ones_like(far)
    s = torch.sigmoid(v)
    return (s + (far * s * torch.sigmoid(-v) * dv).abs()) * (16 + 8 * v.abs().clamp(max=100)) * 2 * U + 2.0 ** -110


def product_bound(length, magnitudes, dtype):
    """What a sum of `length` products loses whose absolute values sum to `magnitudes`.
    fp32: one rounding per fused multiply-add; or three tf32 products, where x = hi + lo with
    |lo| < 2^-10 |x| (hi has 11 bits): lo lo' is left out, below 2^-20 |x x'|, and each lo is read
    to 11 bits, 2^-21 |x| off, twice: 2^-19 = 32 U of each product in all, beside a sum in fp32.
    bf16: the tensor core cuts (does not round) each step of at most 16 products, a step's
    own sum to a few bits below its largest term, so at most two whole fp32 steps per
    product are counted."""
    return (length + 34) * U * magnitudes if dtype == "f32" else (length + 2) * 4 * U * magnitudes


def forward_act(inp, weight, bias, residual, act, dtype):
    """((out, bound), (pre, bound))"""
    pre = inp @ weight.t()
    mag = inp.abs() @ weight.abs().t()
    if bias is not None:
        pre, mag = pre + bias, mag + bias.abs()
    e = product_bound(inp.shape[1], mag, dtype)
    out = act_value(pre, act)
    e_out = 1.13 * e + act_value_bound(pre, act)  # no activation is steeper than 1.13
    if residual is not None:
        out = out + residual
        e_out = e_out + U * out.abs()
    return (out, stored(e_out, out, dtype)), (pre, stored(e, pre, dtype))


def run_act(dout, inp, weight, pre, dweight, act, dtype, splits=16):
    """((dpre, bound), (dweight, bound), (dbias, bound))"""
    p, mag = dout @ weight, dout.abs() @ weight.abs()
    e = product_bound(weight.shape[0], mag, dtype)
    slope, e_slope = act_slope(pre, act), act_slope_bound(pre, act)
    dpre = p * slope
    e_dpre = e * (slope.abs() + e_slope) + p.abs() * e_slope + U * dpre.abs()
    dw = dweight + dout.t() @ inp
    e_dw = product_bound(inp.shape[0] + splits, dout.abs().t() @ inp.abs() + dweight.abs(), dtype)
    db = dout.sum(0)
    e_db = (dout.shape[0] + splits) * U * dout.abs().sum(0)
    return (dpre, stored(e_dpre, dpre, dtype)), (dw, stored(e_dw, dw, dtype)), (db, stored(e_db, db, dtype))


# ------------------------------------------------------------------ norms

def depth(C):
    """Additions that a value goes through in a row's sum (a thread's values, a warp's
    butterfly, a team's warps), at most."""
    return C / 32 + 40


def norm_rows(v, kind, weight, bias, e_v):
    """(y, bound of y, mean, its bound, rstd, its bound, normalised rows) of rows that are
    known to e_v. To first order the normalised row moves by rstd (d - mean d - n mean(n d))
    with a change d of the row; to that come the sums' roundings."""
    if kind == "none":
        return v, e_v, None, None, None, None, v
    C = v.shape[1]
    deep = depth(C)
    mean = v.mean(1, keepdim=True) if kind == "layer" else 0 * v[:, :1]
    e_mean = ((deep + 4) * U * v.abs().mean(1, keepdim=True) + e_v.mean(1, keepdim=True)) if kind == "layer" else 0 * mean
    d = v - mean
    var = d.square().mean(1, keepdim=True)
    rstd = 1 / (var + EPS).sqrt()
    e_d = e_v + e_mean + U * d.abs()
    e_var = (deep + 6) * U * var + 2 * (d.abs() * e_d).mean(1, keepdim=True) + (e_d ** 2).mean(1, keepdim=True)
    e_rstd = rstd * (0.5 * e_var / (var + EPS) * (1 + e_var / (var + EPS)) + 4 * U)
    n = d * rstd
    e_n = e_d * (rstd + e_rstd) + d.abs() * e_rstd + 2 * U * n.abs()
    y = n * weight
    e_y = weight.abs() * e_n + 2 * U * y.abs()
    if bias is not None:
        y = y + bias
        e_y = e_y + 2 * U * y.abs()
    return y, e_y, mean[:, 0], e_mean[:, 0], rstd[:, 0], e_rstd[:, 0], n


def residual_forward(x, branch, gate, wp, bp, w, b, scale, post, norm, dtype):
    """{name: (value, bound)}"""
    z, e_z, mp, e_mp, rp, e_rp, _ = norm_rows(branch, post, wp, bp if post == "layer" else None, 0 * branch)
    g = scale * (torch.ones_like(x[:1]) if gate is None else gate)
    r = x + g * z
    e_r = g.abs() * e_z + 3 * U * ((g * z).abs() + r.abs())
    got = {"residual_out": (r, stored(e_r, r, dtype)), "mean_post": (mp, e_mp), "rstd_post": (rp, e_rp)}
    y, e_y, m, e_m, rs, e_rs, _ = norm_rows(r, norm, w, b if norm == "layer" else None, e_r)
    if norm != "none":
        got["out"] = (y, stored(e_y, y, dtype))
    got["mean"], got["rstd"] = (m, e_m), (rs, e_rs)
    return {k: (v, (None if e is None else e + U * v.abs())) for k, (v, e) in got.items() if v is not None}


def normalised(v, kind, mean, rstd):
    if kind == "none":
        return v
    return (v - (mean[:, None] if kind == "layer" else 0)) * rstd[:, None]


def through_norm(g, n, kind, rstd):
    """(gradient of the row, bound of it / (steps)) from the gradient g of the normalised row."""
    if kind == "none":
        return g, g.abs()
    C = g.shape[1]
    gn = g * n
    out = g - n * gn.mean(1, keepdim=True)
    mag = g.abs() + n.abs() * gn.abs().mean(1, keepdim=True)
    if kind == "layer":
        out = out - g.mean(1, keepdim=True)
        mag = mag + g.abs().mean(1, keepdim=True)
    del C
    return out * rstd[:, None], mag * rstd[:, None]


def residual_backward(dout, dres, res, branch, gate, wp, bp, w, stats, old, scale, post, norm, dtype):
    """{name: (value, bound)}; stats: (mean_post, rstd_post, mean, rstd) as stored; old: the
    parameters' gradients before. `deep` roundings of a row's sum, eight of everything else
    that leads to a value, count on the sum of its terms' magnitudes."""
    mp, rp, m, rs = stats
    shape = branch if branch is not None else res
    C, rows = shape.shape[1], shape.shape[0]
    deep = (depth(C) + 16) * U
    one = torch.ones_like(shape[:1])
    dx, mag = 0 * shape, 0 * shape
    if norm != "none":
        n = normalised(res, norm, m, rs)
        dx, mag = through_norm(dout * w, n, norm, rs)
    if dres is not None:
        dx, mag = dx + dres, mag + dres.abs()
    e_dx = deep * mag
    got = {"dx": (dx, stored(e_dx, dx, dtype))}
    g = scale * (one if gate is None else gate)
    dy, e_dy = g * dx, g.abs() * (e_dx + 2 * U * dx.abs())
    if branch is not None or post == "none":
        z = normalised(branch, post, mp, rp) if branch is not None else None
        gw, e_gw = (dy, e_dy) if post == "none" else (dy * wp, e_dy * wp.abs() + 2 * U * (dy * wp).abs())
        db, mag_db = through_norm(gw, z, post, rp) if post != "none" else (gw, gw.abs())
        e_db = deep * mag_db + (through_norm(e_gw, z.abs(), post, -rp)[1].abs() if post != "none" else e_gw)
        got["dbranch"] = (db, stored(e_db, db, dtype))
    tall = (rows + 64) * U  # roundings of a sum over rows

    def column(name, terms, errs):
        if old.get(name) is not None:
            v = old[name] + terms.sum(0)
            e = tall * (terms.abs().sum(0) + old[name].abs()) + errs.sum(0) + 8 * U * v.abs()
            got[name] = (v, stored(e, v, dtype))

    if norm != "none":
        column("dweight", dout * n, 4 * U * (dout * n).abs())
        column("dbias", dout, 0 * dout)
    if branch is not None:
        y = z if post == "none" else z * wp + (bp if post == "layer" and bp is not None else 0)
        # the sums of dx z and of dx are formed first, the weights come after
        wide = z.abs() if post == "none" else z.abs() * wp.abs() + (bp.abs() if post == "layer" and bp is not None else 0)
        if old.get("dgate") is not None:
            v = old["dgate"] + scale * (dx * y).sum(0)
            e = abs(scale) * (((e_dx + 6 * U * dx.abs()) * wide).sum(0) + tall * (dx.abs() * wide).sum(0)) + tall * old["dgate"].abs()
            got["dgate"] = (v, stored(e, v, dtype))
        if post != "none":
            column("dweight_post", dy * z, e_dy * z.abs() + 6 * U * (dy * z).abs())
    if post == "layer":
        column("dbias_post", dy, e_dy)
    return got
