"""The norms around a block with its gate, scale and residual, on the GPU against 64 bits."""
import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm

pytestmark = pytest.mark.gpu
DT = {"bf16": mm.BF16, "f32": mm.F32}
KIND = {"none": mm.NORM_NONE, "layer": mm.NORM_LAYER, "rms": mm.NORM_RMS}
NAN = float("nan")
STATS = ("mean_post", "rstd_post", "mean", "rstd")
PARAMS = ("dgate", "dweight_post", "dbias_post", "dweight", "dbias")
# widths of every kernel variant, their borders, and ragged ones
WIDTHS = [8, 64, 264, 768, 1024, 1032, 1600, 2048, 2056, 3000, 4096, 4104, 6400, 8192, 8200, 16384, 16392, 32768]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()


def ok(rc):
    assert rc == mm.OK, mm.strerror(rc)


def has(kind, what):
    return kind == "layer" or (kind == "rms" and what != "bias" and what != "mean")


def inputs(T, C, dtype, post, norm, gate=True, seed=0):
    n = lambda k, *s, std=1.0: ref.rounded(ref.normal(seed + k, *s, std=std), dtype)  # noqa: E731
    shift = torch.linspace(-2, 2, T, dtype=torch.float64, device="cuda")[:, None] if T > 1 else 0.5
    x = dict(x=ref.rounded(n(1, T, C) + shift, dtype), branch=ref.rounded(n(2, T, C, std=0.5) - shift, dtype),
             gate=n(3, C) if gate else None)
    for k, kind in (("_post", post), ("", norm)):
        x["weight" + k] = n(4 + len(k), C) + 1 if kind != "none" else None
        x["bias" + k] = n(14 + len(k), C) if kind == "layer" else None
    for k in ("weight_post", "weight"):
        if x[k] is not None:
            x[k] = ref.rounded(x[k], dtype)
    x["dout"] = n(21, T, C) if norm != "none" else None
    x["dresidual"] = n(22, T, C)
    for i, k in enumerate(PARAMS):
        x[k] = n(30 + i, C)
    return x


def dev(v, dtype):
    return None if v is None else v.to(ref.TDT[dtype])


def forward(x, scale, post, norm, dtype, in_place=False, stats=True):
    T, C = x["x"].shape
    d = {k: dev(x[k], dtype) for k in ("x", "branch", "gate", "weight_post", "bias_post", "weight", "bias")}
    out = torch.full((T, C), NAN, device="cuda", dtype=ref.TDT[dtype]) if norm != "none" else None
    r = d["x"] if in_place else torch.full((T, C), NAN, device="cuda", dtype=ref.TDT[dtype])
    s = {k: torch.full((T,), NAN, device="cuda") if stats else None for k in STATS}
    ok(mm.lnbwd_residual_forward(out, r, s["mean_post"], s["rstd_post"], s["mean"], s["rstd"], d["x"], d["branch"], d["gate"],
                                 d["weight_post"], d["bias_post"], d["weight"], d["bias"], 1, T, C, scale, ref.EPS, KIND[post],
                                 KIND[norm], DT[dtype]))
    return {"out": out, "residual_out": r, **s}


def check_forward(x, scale, post, norm, dtype):
    got = forward(x, scale, post, norm, dtype)
    want = ref.residual_forward(x["x"], x["branch"], x["gate"], x["weight_post"], x["bias_post"], x["weight"], x["bias"],
                                torch.tensor(scale).item(), post, norm, dtype)
    for k, (v, e) in want.items():
        if k in STATS and not has(post if k.endswith("post") else norm, k.split("_")[0]):
            continue
        ref.check(got[k], v, e, k)
    for k in STATS:  # what a norm does not have is not written
        if not has(post if k.endswith("post") else norm, k.split("_")[0]):
            assert torch.isnan(got[k]).all(), k
    return got


def backward(x, stats, scale, post, norm, dtype, in_place=False, skip=(), ws=None, residual="x", dresidual=True):
    T, C = x["x"].shape
    d = {k: dev(v, dtype) for k, v in x.items()}
    dres = d["dresidual"] if dresidual else None
    dx = dres if in_place else torch.full((T, C), NAN, device="cuda", dtype=ref.TDT[dtype])
    dbranch = None if "dbranch" in skip else torch.full((T, C), NAN, device="cuda", dtype=ref.TDT[dtype])
    n = mm.lnbwd_residual_backward_workspace_bytes(1, T, C, DT[dtype])
    ws = torch.full((n,), 0xFF, device="cuda", dtype=torch.uint8) if ws is None else ws
    p = [None if k in skip else d[k] for k in PARAMS]
    ok(mm.lnbwd_residual_backward(dx, dbranch, *p, d["dout"], dres, d[residual], d["branch"], d["gate"], d["weight_post"], d["bias_post"],
                                  d["weight"], *[stats.get(k) for k in STATS], ws, n, 1, T, C, scale, KIND[post], KIND[norm], DT[dtype]))
    return {"dx": dx, "dbranch": dbranch, **dict(zip(PARAMS, p))}


def row_statistics(x, post, norm):
    """As the forward stores them: fp32, of the rows given."""
    s = {}
    for k, kind, rows in (("_post", post, x["branch"]), ("", norm, x["x"])):
        mean = rows.mean(1) if kind == "layer" else torch.zeros_like(rows[:, 0])
        s["mean" + k] = mean.float() if kind == "layer" else None
        s["rstd" + k] = (1 / ((rows - mean[:, None]).square().mean(1) + ref.EPS).sqrt()).float() if kind != "none" else None
    return s


def wanted(x, stats, scale, post, norm, dtype, dresidual=True):
    old = {k: x[k] for k in PARAMS}
    if x["gate"] is None:
        old["dgate"] = None
    return ref.residual_backward(x["dout"], x["dresidual"] if dresidual else None, x["x"], x["branch"], x["gate"], x["weight_post"],
                                 x["bias_post"], x["weight"], [None if stats[k] is None else stats[k].double() for k in STATS], old,
                                 torch.tensor(scale).item(), post, norm, dtype)


def check_backward(x, scale, post, norm, dtype):
    s = row_statistics(x, post, norm)
    got = backward(x, s, scale, post, norm, dtype)
    want = wanted(x, s, scale, post, norm, dtype)
    for k, (v, e) in want.items():
        if k == "dbias" and norm != "layer":
            continue
        ref.check(got[k], v, e, k)
    for k in PARAMS:  # what there is no parameter for is left as it was
        absent = {"dgate": x["gate"] is None, "dweight_post": post == "none", "dbias_post": post != "layer", "dweight": norm == "none",
                  "dbias": norm != "layer"}[k]
        if absent:
            assert torch.equal(got[k], dev(x[k], dtype)), k
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(C, dtype):
    T = 13 if C <= 8192 else 5
    x = inputs(T, C, dtype, "layer", "layer", seed=C)
    check_forward(x, 0.5, "layer", "layer", dtype)
    check_backward(x, 0.5, "layer", "layer", dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("norm", ref.KINDS)
@pytest.mark.parametrize("post", ref.KINDS)
def test_kinds(post, norm, gate, dtype):
    for C in (328, 4360):
        x = inputs(9, C, dtype, post, norm, gate, seed=C)
        scale = 1.0 if not gate else -0.3
        got = check_forward(x, scale, post, norm, dtype)
        for again in (forward(x, scale, post, norm, dtype, in_place=True), forward(x, scale, post, norm, dtype, stats=False)):
            assert torch.equal(again["residual_out"], got["residual_out"])
            assert norm == "none" or torch.equal(again["out"], got["out"])
        full = check_backward(x, scale, post, norm, dtype)
        s = row_statistics(x, post, norm)
        again = backward(x, s, scale, post, norm, dtype, in_place=True)
        for k, v in full.items():
            assert torch.equal(again[k], v), k
        for skip in (("dbranch",), PARAMS, ("dgate", "dbranch"), ("dweight_post", "dbias"), ("dbranch", "dgate", "dweight_post"),
                     ("dbranch",) + PARAMS):
            again = backward(x, s, scale, post, norm, dtype, skip=skip)
            for k, v in full.items():
                if k not in skip:
                    assert torch.equal(again[k], v), (skip, k)


@pytest.mark.parametrize("T", [1, 2, 3, 7, 150, 153, 1217, 5000])
def test_rows(T):
    for C, dtype, post, norm in ((520, "bf16", "rms", "rms"), (1600, "bf16", "none", "layer"), (260, "f32", "layer", "rms")):
        x = inputs(T, C, dtype, post, norm, seed=T)
        check_forward(x, 0.7, post, norm, dtype)
        check_backward(x, 0.7, post, norm, dtype)


@pytest.mark.parametrize("post,norm", [("layer", "layer"), ("rms", "rms"), ("none", "layer")])
def test_without_the_residuals_gradient(post, norm):
    x = inputs(21, 264, "bf16", post, norm)
    s = row_statistics(x, post, norm)
    got, want = backward(x, s, 0.5, post, norm, "bf16", dresidual=False), wanted(x, s, 0.5, post, norm, "bf16", dresidual=False)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, k) if not (k == "dbias" and norm != "layer") else None


def test_rows_of_one_value_and_of_zeros():
    """No variance: rstd is 1 / sqrt(eps), the LayerNorm gives its bias."""
    for dtype in ("bf16", "f32"):
        x = inputs(6, 1008, dtype, "layer", "layer", gate=False)
        x["branch"][1], x["branch"][2] = 2.5, 0.0
        x["x"][1], x["x"][2], x["bias_post"][:] = -1.0, 0.0, 0.25
        got = check_forward(x, 1.0, "layer", "layer", dtype)
        for r in (1, 2):  # the residual row is one value too
            assert torch.equal(got["out"][r], dev(x["bias"], dtype))
        check_backward(x, 1.0, "layer", "layer", dtype)


def test_a_large_mean_costs_no_precision():
    x = inputs(8, 768, "f32", "layer", "layer")
    x["branch"] = ref.rounded(x["branch"] + 4096, "f32")
    x["x"] = ref.rounded(x["x"] - 2048, "f32")
    check_forward(x, 1.0, "layer", "layer", "f32")


def test_non_finite_values_stay_in_their_rows():
    for C in (264, 4360):
        x = inputs(12, C, "bf16", "rms", "layer", seed=3)
        s = row_statistics(x, "rms", "layer")
        clean, back = forward(x, 0.5, "rms", "layer", "bf16"), backward(x, s, 0.5, "rms", "layer", "bf16")
        x["branch"][3, 17], x["x"][8, 200] = NAN, float("inf")
        bad = forward(x, 0.5, "rms", "layer", "bf16")
        keep = [i for i in range(12) if i not in (3, 8)]
        for k in ("out", "residual_out", "rstd_post", "mean", "rstd"):
            assert torch.equal(bad[k][keep], clean[k][keep]), k
        assert torch.isnan(bad["out"][[3, 8]]).all()
        x = inputs(12, C, "bf16", "rms", "layer", seed=3)
        x["dout"][5, 9] = NAN
        bad = backward(x, s, 0.5, "rms", "layer", "bf16")
        keep = [i for i in range(12) if i != 5]
        for k in ("dx", "dbranch"):
            assert torch.equal(bad[k][keep], back[k][keep]) and torch.isnan(bad[k][5]).all(), k


def test_nothing_outside_the_outputs_is_written():
    T, C = 11, 1032
    x = inputs(T, C, "bf16", "layer", "layer")
    d = {k: dev(v, "bf16") for k, v in x.items()}
    s = row_statistics(x, "layer", "layer")
    n = mm.lnbwd_residual_backward_workspace_bytes(1, T, C, mm.BF16)
    room = torch.full((9, T * C + 512), 3.0, device="cuda", dtype=torch.bfloat16)
    st = torch.full((4, T + 64), 3.0, device="cuda")
    ws = torch.full((n + 512,), 7, device="cuda", dtype=torch.uint8)
    o = [room[i, 256:] for i in range(9)]
    ok(mm.lnbwd_residual_forward(o[0], o[1], *[st[i, 32:] for i in range(4)], d["x"], d["branch"], d["gate"], d["weight_post"],
                                 d["bias_post"], d["weight"], d["bias"], 1, T, C, 1.0, ref.EPS, 1, 1, mm.BF16))
    ok(mm.lnbwd_residual_backward(o[2], o[3], *o[4:9], d["dout"], d["dresidual"], d["x"], d["branch"], d["gate"], d["weight_post"],
                                  d["bias_post"], d["weight"], *[s[k] for k in STATS], ws[256:], n, 1, T, C, 1.0, 1, 1, mm.BF16))
    torch.cuda.synchronize()
    assert (room[:, :256] == 3).all() and (room[:4, 256 + T * C:] == 3).all() and (room[4:, 256 + C:] == 3).all()
    assert (st[:, :32] == 3).all() and (st[:, 32 + T:] == 3).all()
    assert (ws[:256] == 7).all() and (ws[256 + n:] == 7).all()


def test_empty_calls():
    for T, C in ((0, 64), (5, 0)):
        ok(mm.lnbwd_residual_forward(*[None] * 13, 1, T, C, 1.0, 1e-5, 1, 1, mm.F32))
        assert mm.lnbwd_residual_backward_workspace_bytes(1, T, C, mm.F32) == 0
        ok(mm.lnbwd_residual_backward(*[None] * 20, 0, 1, T, C, 1.0, 1, 1, mm.F32))


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits along random directions (errors of
    order 1e-8 and 1e-12) against the fp32 gradients from the fp32 forward's own outputs,
    off by some tens of 2^-24 of the terms' magnitudes: 1e-4 of the norms' product."""
    T, C, scale = 17, 48, 0.6
    for post, norm in (("layer", "layer"), ("rms", "rms"), ("layer", "rms"), ("none", "layer")):
        x = inputs(T, C, "f32", post, norm, seed=1)
        names = [k for k in ("x", "branch", "gate", "weight_post", "bias_post", "weight", "bias") if x[k] is not None]

        def loss(v):
            v = {**x, **v}
            got = ref.residual_forward(v["x"], v["branch"], v["gate"], v["weight_post"], v["bias_post"], v["weight"], v["bias"], scale,
                                       post, norm, "f32")
            return ((got["residual_out"][0] * x["dresidual"]).sum() + (got["out"][0] * x["dout"]).sum()).item()

        fwd = forward(x, scale, post, norm, "f32")
        zero = {**x, **{k: torch.zeros(C, device="cuda", dtype=torch.float64) for k in PARAMS}, "r": fwd["residual_out"].double()}
        got = backward(zero, fwd, scale, post, norm, "f32", residual="r")
        for i, k in enumerate(names):
            d = ref.normal(60 + i, *x[k].shape)
            h = 1e-4
            slope = (loss({k: x[k] + h * d}) - loss({k: x[k] - h * d})) / (2 * h)
            g = got["d" + k].double()
            assert abs(slope - (g * d).sum().item()) <= 1e-4 * (g.norm() * d.norm()).item(), (post, norm, k)


def test_captured_replayed_and_repeated():
    T, C = 333, 1600
    x, y = (inputs(T, C, "bf16", "rms", "layer", seed=k) for k in (1, 100))
    d = {k: dev(v, "bf16") for k, v in x.items()}
    st = {k: torch.empty(T, device="cuda") for k in STATS}
    r, out, dx, db = (torch.empty_like(d["x"]) for _ in range(4))
    n = mm.lnbwd_residual_backward_workspace_bytes(1, T, C, mm.BF16)
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)

    def calls(w):
        ok(mm.lnbwd_residual_forward(out, r, *[st[k] for k in STATS], d["x"], d["branch"], d["gate"], d["weight_post"], None,
                                     d["weight"], d["bias"], 1, T, C, 0.5, ref.EPS, 2, 1, mm.BF16))
        ok(mm.lnbwd_residual_backward(dx, db, *[d[k] for k in PARAMS], d["dout"], d["dresidual"], r, d["branch"], d["gate"],
                                      d["weight_post"], None, d["weight"], *[st[k] for k in STATS], w, n, 1, T, C, 0.5, 2, 1, mm.BF16))

    calls(torch.empty_like(ws))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        calls(ws)
    every = lambda: [t.clone() for t in (r, out, dx, db, *st.values(), *[d[k] for k in PARAMS])]  # noqa: E731
    seen = []
    for again in (graph.replay, lambda: calls(torch.empty_like(ws)), graph.replay):
        for k, v in y.items():
            if v is not None:
                d[k].copy_(dev(v, "bf16"))
        for t in (r, out, dx, db):
            t.fill_(NAN)
        torch.cuda.synchronize()
        again()
        torch.cuda.synchronize()
        seen.append(every())
    for a, b, c in zip(*seen):
        assert torch.equal(a.nan_to_num(-7), b.nan_to_num(-7)) and torch.equal(a.nan_to_num(-7), c.nan_to_num(-7))


def test_two_streams_with_workspaces_of_their_own():
    xs = [inputs(700, 768, "bf16", "layer", "layer", seed=200 * i) for i in range(2)]
    stats = [row_statistics(x, "layer", "layer") for x in xs]
    want = [backward(x, s, 0.5, "layer", "layer", "bf16") for x, s in zip(xs, stats)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                s.wait_stream(torch.cuda.default_stream())
                got[i].append(backward(xs[i], stats[i], 0.5, "layer", "layer", "bf16"))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for k, v in want[i].items():
                assert torch.equal(g[k], v), k


def test_failed_launches_and_host_memory():
    x = inputs(4, 64, "f32", "layer", "layer")
    d = {k: dev(v, "f32") for k, v in x.items()}
    r = torch.full((4, 64), 9.0, device="cuda")
    args = [None] * 4 + [d["x"], d["branch"], d["gate"], d["weight_post"], d["bias_post"], d["weight"], d["bias"], 1, 4, 64, 1.0, 1e-5, 1, 1, mm.F32]
    mm.mmbwd_debug_fail_next_launch(1)
    assert mm.lnbwd_residual_forward(torch.empty_like(r), r, *args) == mm.ERR_CUDA
    torch.cuda.synchronize()
    assert (r == 9).all()
    args[5] = torch.zeros(4, 64)
    assert mm.lnbwd_residual_forward(torch.empty_like(r), r, *args) == mm.ERR_MEMORY


def test_offsets_beyond_32_bits():
    """More than 2^31 values, rows that repeat 997 different ones: both ends against 64 bits,
    and every repetition the same."""
    T, C = 530_000, 4104
    x = inputs(997, C, "bf16", "rms", "layer", seed=7)
    many = lambda t: dev(t, "bf16").repeat(T // 997 + 1, 1)[:T].contiguous()  # noqa: E731
    d = {k: dev(x[k], "bf16") for k in ("gate", "weight_post", "weight", "bias")}
    r, branch = many(x["x"]), many(x["branch"])
    s = {k: torch.full((T,), NAN, device="cuda") if k != "mean_post" else None for k in STATS}
    out = torch.full((T, C), NAN, device="cuda", dtype=torch.bfloat16)
    ok(mm.lnbwd_residual_forward(out, r, *s.values(), r, branch, d["gate"], d["weight_post"], None, d["weight"], d["bias"], 1, T, C, 0.5,
                                 ref.EPS, mm.NORM_RMS, mm.NORM_LAYER, mm.BF16))
    want = ref.residual_forward(x["x"], x["branch"], x["gate"], x["weight_post"], None, x["weight"], x["bias"], 0.5, "rms", "layer", "bf16")
    got = {"out": out, "residual_out": r, **s}
    rows = torch.tensor([*range(20), *range(T - 300, T)], device="cuda")
    for k, (v, e) in want.items():
        if k != "mean_post":
            ref.check(got[k][rows], v[rows % 997], e[rows % 997], k)
            for i in range(0, T - 997, 997):
                assert torch.equal(got[k][i:i + 997], got[k][:997]), (k, i)
    dres = many(x["dresidual"])
    dout = torch.zeros_like(dres)
    dout[T - 300:] = dev(x["dout"], "bf16")[rows[20:] % 997]
    dbranch = out
    dbias = torch.zeros(C, device="cuda", dtype=torch.bfloat16)
    n = mm.lnbwd_residual_backward_workspace_bytes(1, T, C, mm.BF16)
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    ok(mm.lnbwd_residual_backward(dres, dbranch, None, None, None, None, dbias, dout, dres, r, branch, d["gate"], d["weight_post"], None,
                                  d["weight"], *s.values(), ws, n, 1, T, C, 0.5, mm.NORM_RMS, mm.NORM_LAYER, mm.BF16))
    stats = [None if s[k] is None else s[k][rows].double() for k in STATS]
    want = ref.residual_backward(dout[rows].double(), x["dresidual"][rows % 997], r[rows].double(), x["branch"][rows % 997], x["gate"],
                                 x["weight_post"], None, x["weight"], stats, {}, 0.5, "rms", "layer", "bf16")
    ref.check(dres[rows], *want["dx"], "dx")
    ref.check(dbranch[rows], *want["dbranch"], "dbranch")
    for i in range(0, T - 300 - 997, 997):
        assert torch.equal(dres[i:i + 997], dres[:997]) and torch.equal(dbranch[i:i + 997], dbranch[:997]), i
    total = dout[T - 300:].double()
    e = 400 * ref.U * total.abs().sum(0)  # (zeros add without a rounding)
    ref.check(dbias, total.sum(0), ref.stored(e, total.sum(0), "bf16"), "dbias")
