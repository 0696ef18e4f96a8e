"""The linear layer with an activation and a residual in its epilogue, and the gradients
through the activation, on the GPU against 64 bits."""
import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm

pytestmark = pytest.mark.gpu
DT = {"bf16": mm.BF16, "f32": mm.F32}
ACT = {"none": mm.ACT_NONE, "gelu": mm.ACT_GELU, "silu": mm.ACT_SILU, "relu": mm.ACT_RELU}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()


@pytest.fixture(autouse=True)
def no_failed_wait():
    yield
    torch.cuda.synchronize()
    assert mm.mmbwd_device_status()[0] == mm.OK


def ok(rc):
    assert rc == mm.OK, mm.strerror(rc)


def inputs(T, C, OC, dtype, seed=0, bias=True, residual=True):
    n = lambda k, *s, std=1.0: ref.rounded(ref.normal(seed + k, *s, std=std), dtype)  # noqa: E731
    return dict(inp=n(1, T, C), weight=n(2, OC, C, std=max(C, 1) ** -0.5), bias=n(3, OC) if bias else None,
                residual=n(4, T, OC) if residual else None)


def dev(x, dtype):
    return None if x is None else x.to(ref.TDT[dtype])


def forward(x, act, dtype, pre=True, in_place=False):
    T, C = x["inp"].shape
    OC = x["weight"].shape[0]
    d = {k: dev(v, dtype) for k, v in x.items()}
    out = d["residual"] if in_place else torch.full((T, OC), NAN, device="cuda", dtype=ref.TDT[dtype])
    p = torch.full_like(out, NAN) if pre else None
    ok(mm.mmbwd_forward_act(out, p, d["inp"], d["weight"], d["bias"], d["residual"], 1, T, C, OC, ACT[act], DT[dtype]))
    return out, p


def check_forward(x, act, dtype, **kw):
    out, pre = forward(x, act, dtype, **kw)
    want, want_pre = ref.forward_act(x["inp"], x["weight"], x["bias"], x["residual"], act, dtype)
    ref.check(out, *want, "out")
    if pre is not None:
        ref.check(pre, *want_pre, "pre")
    return out, pre


# tokens around every kernel's rows and tiles; widths that end inside a tile, a k-block or a vector
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 16, 17, 31, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("size", [(8, 8), (64, 200), (136, 1000), (1600, 264), (2056, 72)], ids=lambda s: "x".join(map(str, s)))
def test_forward_sizes(T, size, dtype):
    check_forward(inputs(T, *size, dtype), "gelu", dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 40, 260])
@pytest.mark.parametrize("act", ref.ACTS)
def test_forward_activations_and_options(act, T, dtype):
    for bias in (True, False):
        for residual in (True, False):
            x = inputs(T, 328, 264, dtype, 9, bias, residual)
            full = check_forward(x, act, dtype)[0]
            assert torch.equal(forward(x, act, dtype, pre=False)[0], full)  # pre changes nothing
            if residual:
                assert torch.equal(forward(x, act, dtype, in_place=True)[0], full)
                assert torch.equal(forward(x, act, dtype, pre=False, in_place=True)[0], full)


@pytest.mark.parametrize("T,C,OC", [(4100, 1600, 1608), (1000, 264, 6408), (48, 6400, 1600), (1, 6400, 50304), (6, 12800, 40)])
def test_forward_many_tiles(T, C, OC):
    """Several items to each CTA pair, ragged at both ends; long rows of few tokens."""
    check_forward(inputs(T, C, OC, "bf16", 3), "silu", "bf16")


def test_forward_long_sum_f32():
    """A reduction beyond 8192 of operands of one sign, where a sum that is cut instead of rounded shows."""
    for T in (4, 100):
        x = inputs(T, 9000, 40, "f32", 4)
        x["inp"], x["weight"] = x["inp"].abs(), x["weight"].abs()
        check_forward(x, "none", "f32")


@pytest.mark.parametrize("path", ["32", "64", "spans"])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("size", [(1, 4, 4), (33, 100, 36), (65, 264, 1300), (300, 772, 132), (1030, 1156, 392)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fp32_kernels(monkeypatch, size, act, path):
    """Each fp32 kernel, forward and backward, at sizes that end inside its tiles and spans."""
    monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)
    for options in (dict(), dict(bias=False, residual=False)):
        x = inputs(*size, "f32", 21, **options)
        full = check_forward(x, act, "f32")[0]
        assert torch.equal(forward(x, act, "f32", pre=False)[0], full)
        if x["residual"] is not None:
            assert torch.equal(forward(x, act, "f32", in_place=True)[0], full)
    x = gradient_inputs(*size, "f32", act, 22)
    full = check_run(x, act, "f32")
    for a, b in zip(run(x, act, "f32", bias=False)[:2] + run(x, act, "f32", in_place=True), full[:2] + full):
        assert torch.equal(a, b)


@pytest.mark.parametrize("path", ["32", "spans"])
def test_fp32_long_sums_of_one_sign(monkeypatch, path):
    """Reductions of 9000 and 5000 values of one sign: a sum that is cut instead of rounded
    loses 2^-24 of itself a step and would be over the bound of 2-norms (2e-6: a random walk of 9000
    roundings is 95 steps of 2^-24 on the last sums, 6e-6 at the very most, a third of that on
    average over the way there)."""
    monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)
    x = inputs(100, 9000, 40, "f32", 4, bias=False, residual=False)
    x["inp"], x["weight"] = x["inp"].abs(), x["weight"].abs()
    out = forward(x, "none", "f32")[0].double()
    want = x["inp"] @ x["weight"].t()
    assert (out - want).norm() <= 2e-6 * want.norm()
    check_forward(x, "none", "f32")


def test_fp32_many_items(monkeypatch):
    monkeypatch.setenv("MMBWD_ACT_F32_PATH", "spans")
    check_forward(inputs(3000, 520, 2052, "f32", 23), "gelu", "f32")
    check_run(gradient_inputs(2600, 1604, 1000, "f32", "gelu", 24), "gelu", "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_inputs(dtype):
    """C == 0: the activation of the bias, over every kind of value."""
    vals = torch.cat([torch.linspace(-30, 30, 2001, dtype=torch.float64), torch.tensor([1e-30, -1e-30, 1e10, -1e10, 1e30, -1e30, 0.0]),
                      torch.logspace(-6, 3, 992, dtype=torch.float64), -torch.logspace(-6, 3, 1000, dtype=torch.float64)]).cuda()
    bias = ref.rounded(vals[: vals.numel() // 8 * 8], dtype)
    x = dict(inp=torch.empty(3, 0, device="cuda", dtype=torch.float64), weight=torch.empty(bias.numel(), 0, device="cuda", dtype=torch.float64),
             bias=bias, residual=None)
    for act in ref.ACTS:
        out, pre = check_forward(x, act, dtype)
        assert torch.equal(pre, dev(bias, dtype).expand(3, -1))
    x["bias"], x["residual"] = None, ref.rounded(ref.normal(5, 3, bias.numel()), dtype)
    out, pre = forward(x, "silu", dtype)
    assert torch.equal(out, dev(x["residual"], dtype)) and not pre.any()


def test_empty_calls():
    t = torch.zeros(8, 64, device="cuda")
    for T, OC in ((0, 64), (8, 0)):
        ok(mm.mmbwd_forward_act(t if T and OC else None, None, t if T else None, t if OC else None, None, None, 1, T, 64, OC, 1, mm.F32))
    ok(mm.mmbwd_act_backward(None, None, None, 0, 1, mm.BF16))
    assert not t.any()


def test_non_finite_values_stay_in_their_rows():
    for T in (7, 200):
        x = inputs(T, 264, 136, "bf16", 6)
        clean = forward(x, "gelu", "bf16")[0]
        x["inp"][3, 17], x["inp"][5, 200] = NAN, float("inf")
        bad = forward(x, "gelu", "bf16")[0]
        keep = [i for i in range(T) if i not in (3, 5)]
        assert torch.equal(clean[keep], bad[keep])
        assert torch.isnan(bad[3]).all()
        x["residual"][6, 2] = NAN
        assert torch.isnan(forward(x, "relu", "bf16")[0]).sum() >= 1 and torch.isnan(forward(x, "relu", "bf16")[0][6]).sum() == 1


@pytest.mark.parametrize("T", [3, 30, 300])
def test_nothing_outside_the_outputs_is_written(T):
    C, OC = 72, 136
    x = inputs(T, C, OC, "bf16", 7)
    d = {k: dev(v, "bf16") for k, v in x.items()}
    room = torch.full((3, T * OC + 512), 3.0, device="cuda", dtype=torch.bfloat16)
    out, pre = room[0, 256:256 + T * OC], room[1, 256:256 + T * OC]
    ok(mm.mmbwd_forward_act(out, pre, d["inp"], d["weight"], d["bias"], d["residual"], 1, T, C, OC, 1, mm.BF16))
    assert (room[:2, :256] == 3).all() and (room[:2, 256 + T * OC:] == 3).all()


# ------------------------------------------------------------------ backward

def gradient_inputs(T, C, OC, dtype, act, seed=0):
    n = lambda k, *s, std=1.0: ref.rounded(ref.normal(seed + k, *s, std=std), dtype)  # noqa: E731
    pre = n(1, T, C, std=2.0)
    return dict(dout=n(2, T, OC, std=0.1), weight=n(3, OC, C, std=0.1), pre=pre, inp=ref.rounded(ref.act_value(pre, act), dtype),
                dweight=n(4, OC, C))


def workspace(T, C, OC, dtype):
    n = mm.mmbwd_run_act_workspace_bytes(1, T, C, OC, DT[dtype])
    return torch.full((n,), 0xFF, device="cuda", dtype=torch.uint8) if n else None, n


def run(x, act, dtype, bias=True, in_place=False):
    T, C = x["pre"].shape
    OC = x["weight"].shape[0]
    d = {k: dev(v, dtype) for k, v in x.items()}
    dpre = d["pre"] if in_place else torch.full((T, C), NAN, device="cuda", dtype=ref.TDT[dtype])
    dbias = torch.full((OC,), NAN, device="cuda", dtype=ref.TDT[dtype]) if bias else None
    ws, n = workspace(T, C, OC, dtype)
    ok(mm.mmbwd_run_act(dpre, d["dweight"], dbias, d["dout"], d["inp"], d["weight"], d["pre"], ws, n, 1, T, C, OC, ACT[act], DT[dtype]))
    return dpre, d["dweight"], dbias


def check_run(x, act, dtype):
    got = run(x, act, dtype)
    want = ref.run_act(x["dout"], x["inp"], x["weight"], x["pre"], x["dweight"], act, dtype)
    for name, g, w in zip(("dpre", "dweight", "dbias"), got, want):
        ref.check(g, *w, name)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 8, 8), (5, 64, 200), (63, 264, 136), (300, 520, 72), (129, 2056, 264)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ref.ACTS)
def test_run_sizes(act, size, dtype):
    x = gradient_inputs(*size, dtype, act)
    full = check_run(x, act, dtype)
    for a, b in zip(run(x, act, dtype, bias=False)[:2] + run(x, act, dtype, in_place=True), full[:2] + full):
        assert torch.equal(a, b)


@pytest.mark.parametrize("splits", ["1", "3"])
def test_run_many_items(monkeypatch, splits):
    monkeypatch.setenv("MMBWD_SPLITK", splits)
    check_run(gradient_inputs(3000, 1608, 1000, "bf16", "gelu", 5), "gelu", "bf16")


def test_run_degenerate_sizes():
    d = lambda *s: torch.full(s, 5.0, device="cuda")  # noqa: E731
    dpre, dw, db = d(8, 64), d(16, 64), d(16)
    ok(mm.mmbwd_run_act(dpre, None, None, None, dpre.clone(), None, d(8, 64), None, 0, 1, 8, 64, 0, 1, mm.F32))
    assert not dpre.any()  # the empty sum
    ok(mm.mmbwd_run_act(None, dw, db, None, None, d(16, 64), None, None, 0, 1, 0, 64, 16, 1, mm.F32))
    assert not db.any() and (dw == 5).all()
    ok(mm.mmbwd_run_act(None, None, db, d(8, 16), None, None, None, None, 0, 1, 8, 0, 16, 1, mm.F32))
    assert (db == 40).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ref.ACTS)
def test_alone(act, dtype):
    """Every kind of argument; any number of values; in place over either input."""
    special = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), 1e30, -1e30, 1e-40, NAN, 88.0, -88.0, 10.0, -10.0], dtype=torch.float64)
    pre = ref.rounded(torch.cat([special, torch.linspace(-25, 25, 12289, dtype=torch.float64)]).cuda(), dtype)
    dout = ref.rounded(ref.normal(8, pre.numel()), dtype)
    slope, e = ref.act_slope(pre, act), ref.act_slope_bound(pre, act)
    want = dout * slope
    bound = ref.stored(dout.abs() * e + 2 * ref.U * want.abs(), want, dtype).nan_to_num(0)
    for n in (1, 3, 7, 8, 9, 4095, 4097, pre.numel()):
        p, d = dev(pre[:n], dtype), dev(dout[:n], dtype)
        out = torch.full((n + 64,), 7.0, device="cuda", dtype=ref.TDT[dtype])
        ok(mm.mmbwd_act_backward(out, d, p, n, ACT[act], DT[dtype]))
        ref.check(out[:n], want[:n], bound[:n], f"n={n}")
        assert (out[n:] == 7).all()
        over_d, over_p = d.clone(), p.clone()
        ok(mm.mmbwd_act_backward(over_d, over_d, p, n, ACT[act], DT[dtype]))
        ok(mm.mmbwd_act_backward(over_p, d, over_p, n, ACT[act], DT[dtype]))
        for o in (over_d, over_p):
            assert torch.equal(o.view(torch.int16 if dtype == "bf16" else torch.int32), out[:n].view(torch.int16 if dtype == "bf16" else torch.int32))


def test_gradients_against_differences():
    """The loss sum(out * a) of the layer fc -> act -> projection, moved along random
    directions: central differences of the definition in 64 bits (error of order h^2 = 1e-8
    and of roundings 1e-16 / h = 1e-12) against the fp32 gradients, whose error is a few
    2^-24 of the terms' magnitudes: 1e-4 of their norms leaves room for both."""
    T, C, H, OC = 37, 24, 40, 16
    n = lambda k, *s, std=1.0: ref.rounded(ref.normal(k, *s, std=std), "f32")  # noqa: E731
    x, w1, b1, w2, b2, r, a = n(1, T, C), n(2, H, C, std=0.3), n(3, H), n(4, OC, H, std=0.3), n(5, OC), n(6, T, OC), n(7, T, OC)
    f = lambda t: t.float()  # noqa: E731
    for act in ("gelu", "silu"):
        def loss(x, w1, b1, w2, b2):
            return ((ref.act_value(x @ w1.t() + b1, act) @ w2.t() + b2 + r) * a).sum().item()

        h, pre, out = (torch.empty(T, k, device="cuda") for k in (H, H, OC))
        ok(mm.mmbwd_forward_act(h, pre, f(x), f(w1), f(b1), None, 1, T, C, H, ACT[act], mm.F32))
        ok(mm.mmbwd_forward_act(out, None, h, f(w2), f(b2), f(r), 1, T, H, OC, mm.ACT_NONE, mm.F32))
        dpre, dw2, db2 = torch.empty(T, H, device="cuda"), torch.zeros(OC, H, device="cuda"), torch.empty(OC, device="cuda")
        ok(mm.mmbwd_run_act(dpre, dw2, db2, f(a), h, f(w2), pre, None, 0, 1, T, H, OC, ACT[act], mm.F32))
        dx, dw1, db1 = torch.zeros(T, C, device="cuda"), torch.zeros(H, C, device="cuda"), torch.empty(H, device="cuda")
        ok(mm.mmbwd_run(dx, dw1, db1, dpre, f(x), f(w1), 1, T, C, H, mm.F32))
        # the same dpre with the activation's gradient by itself
        dh = torch.zeros(T, H, device="cuda")
        ok(mm.mmbwd_run(dh, torch.zeros_like(dw2), None, f(a), h, f(w2), 1, T, H, OC, mm.F32))
        ok(mm.mmbwd_act_backward(dh, dh, pre, T * H, ACT[act], mm.F32))
        assert (dh - dpre).norm() <= 1e-5 * dpre.norm()
        leaves, grads = [x, w1, b1, w2, b2], [dx, dw1, db1, dw2, db2]
        for i, (v, g) in enumerate(zip(leaves, grads)):
            d = ref.normal(20 + i, *v.shape)
            step = 1e-4
            up = loss(*[t + step * d if j == i else t for j, t in enumerate(leaves)])
            down = loss(*[t - step * d if j == i else t for j, t in enumerate(leaves)])
            got = (g.double() * d).sum().item()
            assert abs((up - down) / (2 * step) - got) <= 1e-4 * (g.double().norm() * d.norm()).item(), (act, i)


# ------------------------------------------------------------------ streams, graphs, threads

def test_captured_and_replayed_with_new_inputs(monkeypatch):
    monkeypatch.setenv("MMBWD_SPLITK", "2")
    T, C, OC = 300, 264, 392
    x, y = gradient_inputs(T, C, OC, "bf16", "gelu", 1), gradient_inputs(T, C, OC, "bf16", "gelu", 50)
    d = {k: dev(v, "bf16") for k, v in x.items()}
    dpre, db = torch.empty_like(d["pre"]), torch.empty(OC, device="cuda", dtype=torch.bfloat16)
    out, pre, back = torch.empty_like(d["dout"]), torch.empty_like(d["dout"]), torch.empty_like(d["dout"])
    ws, n = workspace(T, C, OC, "bf16")
    ws2 = torch.empty_like(ws)

    def calls(w, dw):
        ok(mm.mmbwd_run_act(dpre, dw, db, d["dout"], d["inp"], d["weight"], d["pre"], w, n, 1, T, C, OC, mm.ACT_GELU, mm.BF16))
        ok(mm.mmbwd_forward_act(out, pre, dpre, d["weight"], db, d["dout"], 1, T, C, OC, mm.ACT_SILU, mm.BF16))
        ok(mm.mmbwd_act_backward(back, d["dout"], pre, T * OC, mm.ACT_SILU, mm.BF16))

    dw = d["dweight"]
    calls(ws2, dw.clone())
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        calls(ws, dw)
    for k, v in y.items():
        d[k].copy_(dev(v, "bf16"))
    dw2 = dw.clone()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (dpre, dw, db, out, pre, back)]
    calls(ws2, dw2)
    torch.cuda.synchronize()
    for a, b in zip(got, (dpre, dw2, db, out, pre, back)):
        assert torch.equal(a, b)


def test_two_streams_with_workspaces_of_their_own(monkeypatch):
    monkeypatch.setenv("MMBWD_SPLITK", "4")
    T, C, OC = 1000, 264, 392
    xs = [gradient_inputs(T, C, OC, "bf16", "silu", 70 * i) for i in range(2)]
    want = [run(x, "silu", "bf16") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    sets = []
    for x in xs:
        d = {k: dev(v, "bf16") for k, v in x.items()}
        sets.append((d, torch.empty_like(d["pre"]), torch.empty(OC, device="cuda", dtype=torch.bfloat16), *workspace(T, C, OC, "bf16")))
    torch.cuda.synchronize()
    for _ in range(20):
        for (d, dpre, db, ws, n), s in zip(sets, streams):
            ok(mm.mmbwd_run_act(dpre, d["dweight"], db, d["dout"], d["inp"], d["weight"], d["pre"], ws, n, 1, T, C, OC, mm.ACT_SILU,
                                mm.BF16, stream=s.cuda_stream))
    torch.cuda.synchronize()
    for (d, dpre, db, _, _), w in zip(sets, want):
        assert torch.equal(dpre, w[0]) and torch.equal(db, w[2])


def test_repeats_are_identical_and_failed_launches_write_nothing():
    x = gradient_inputs(500, 264, 136, "bf16", "gelu", 11)
    first = run(x, "gelu", "bf16")
    for _ in range(3):
        for a, b in zip(run(x, "gelu", "bf16"), first):
            assert torch.equal(a, b)
    for T in (4, 200):
        for dtype in ("bf16", "f32"):
            y = inputs(T, 64, 64, dtype)
            d = {k: dev(v, dtype) for k, v in y.items()}
            out = torch.full((T, 64), 9.0, device="cuda", dtype=ref.TDT[dtype])
            mm.mmbwd_debug_fail_next_launch(1)
            assert mm.mmbwd_forward_act(out, None, d["inp"], d["weight"], None, None, 1, T, 64, 64, 1, DT[dtype]) == mm.ERR_CUDA
            mm.mmbwd_debug_fail_next_launch(1)
            assert mm.mmbwd_act_backward(out, d["inp"], d["inp"], T * 64, 1, DT[dtype]) == mm.ERR_CUDA
            torch.cuda.synchronize()
            assert (out == 9).all()
    host = torch.zeros(64, 64)
    assert mm.mmbwd_act_backward(d["inp"], host, d["inp"], 64, 1, mm.F32) == mm.ERR_MEMORY


# ------------------------------------------------------------------ long lists of items, offsets beyond 32 bits

def rows_of(T):
    """Rows at both ends and around the middle."""
    return sorted({*range(min(T, 70)), *range(T // 2 - 40, T // 2 + 40), *range(max(T - 300, 0), T)})


def tall(T, n, dtype, k):
    """T rows that repeat 997 different ones."""
    few = ref.rounded(ref.normal(k, 997, n), dtype)
    return few, few.to(ref.TDT[dtype]).repeat(T // 997 + 1, 1)[:T].contiguous()


@pytest.mark.parametrize("dtype,T,OC", [("bf16", 66_000, 4096), ("bf16", 530_000, 4104), ("f32", 530_000, 4100)])
def test_forward_of_many_rows(dtype, T, OC):
    """More tiles than a launch's item table holds; more than 2^31 outputs."""
    C = 16
    few, inp = tall(T, C, dtype, 1)
    x = inputs(1, C, OC, dtype, 2, residual=False)
    d = {k: dev(v, dtype) for k, v in x.items()}
    out = torch.full((T, OC), NAN, device="cuda", dtype=ref.TDT[dtype])
    pre = torch.full_like(out, NAN)
    ok(mm.mmbwd_forward_act(out, pre, inp, d["weight"], d["bias"], None, 1, T, C, OC, mm.ACT_GELU, DT[dtype]))
    rows = torch.tensor(rows_of(T), device="cuda")
    for got, want in zip((out, pre), ref.forward_act(few, x["weight"], x["bias"], None, "gelu", dtype)):
        ref.check(got[rows], want[0][rows % 997], want[1][rows % 997])
        for i in range(0, T - 997, 997):  # equal rows in, equal rows out
            assert torch.equal(got[i:i + 997], got[:997]), i
    # in place, from the residual
    ok(mm.mmbwd_forward_act(out, None, inp, d["weight"], d["bias"], out, 1, T, C, OC, mm.ACT_GELU, DT[dtype]))
    first = ref.forward_act(few, x["weight"], x["bias"], ref.rounded(ref.act_value(pre[:997].double(), "gelu"), dtype), "gelu", dtype)[0]
    # (what was added is known to a step of its type, which the sum keeps)
    ref.check(out[rows], first[0][rows % 997], (first[1] + 4 * ref.HALF[dtype] * first[0].abs().clamp(min=1))[rows % 997])


@pytest.mark.parametrize("dtype,T,C", [("bf16", 66_000, 4096), ("bf16", 530_000, 4104), ("f32", 530_000, 4100)])
def test_gradients_of_many_rows(dtype, T, C):
    OC = 16
    dout_few, dout = tall(T, OC, dtype, 3)
    pre_few, dpre = tall(T, C, dtype, 4)
    weight = ref.rounded(ref.normal(5, OC, C, std=0.1), dtype)
    inp = torch.zeros_like(dpre)
    inp[T - 1] = 2.0
    dweight = torch.zeros(OC, C, device="cuda", dtype=ref.TDT[dtype])
    ws, n = workspace(T, C, OC, dtype)
    ok(mm.mmbwd_run_act(dpre, dweight, None, dout, inp, dev(weight, dtype), dpre, ws, n, 1, T, C, OC, mm.ACT_SILU, DT[dtype]))
    (want, bound), _, _ = ref.run_act(dout_few, 0 * pre_few, weight, pre_few, 0 * weight, "silu", dtype)
    rows = torch.tensor(rows_of(T), device="cuda")
    ref.check(dpre[rows], want[rows % 997], bound[rows % 997])
    for i in range(0, T - 997, 997):
        assert torch.equal(dpre[i:i + 997], dpre[:997]), i
    # One product beside zeros, which add without a rounding: exact in bf16. In fp32 hi * 2 + lo * 2,
    # where lo (13 bits of x, below 2^-10 |x|) is read to 11 bits: the bound of one product.
    want = (2 * dout[T - 1]).double()[:, None].expand(OC, C)
    ref.check(dweight, want, ref.product_bound(1, want.abs(), "f32") if dtype == "f32" else 0 * want, "dweight")


def test_alone_beyond_32_bits():
    n = 2 ** 31 + 8 * 12345 + 3
    pre = torch.full((n,), 1.0, device="cuda", dtype=torch.bfloat16)
    dout = torch.full_like(pre, 2.0)
    pre[-5:] = -1.0
    ok(mm.mmbwd_act_backward(dout, dout, pre, n, mm.ACT_RELU, mm.BF16))
    assert (dout[-5:] == 0).all() and (dout[:-5] == 2).all()


@pytest.mark.parametrize("OC", [264, 392])
def test_bias_gradient_by_a_product_of_ones(monkeypatch, OC):
    x = gradient_inputs(600, 520, OC, "bf16", "gelu", 31)
    plain = check_run(x, "gelu", "bf16")
    monkeypatch.setenv("MMBWD_DBIAS", "ones")
    for splits in ("1", "2"):
        monkeypatch.setenv("MMBWD_SPLITK", splits)
        check_run(x, "gelu", "bf16")
    assert plain[0].numel()


@pytest.mark.parametrize("shift", [8, 16, 24])
@pytest.mark.parametrize("T", [20, 300])
def test_rows_that_start_between_32_byte_boundaries(T, shift):
    """Outputs, residual and pre 16-byte aligned, in rows that are multiples of 32 bytes."""
    C, OC = 136, 272
    x = inputs(T, C, OC, "bf16", 41)
    want = check_forward(x, "silu", "bf16")
    d = {k: dev(v, "bf16") for k, v in x.items()}
    room = torch.full((3, T * OC + 64), 3.0, device="cuda", dtype=torch.bfloat16)
    out, pre, res = (r[shift:shift + T * OC].view(T, OC) for r in room)
    res.copy_(d["residual"])
    ok(mm.mmbwd_forward_act(out, pre, d["inp"], d["weight"], d["bias"], res, 1, T, C, OC, mm.ACT_SILU, mm.BF16))
    ok(mm.mmbwd_forward_act(res, None, d["inp"], d["weight"], d["bias"], res, 1, T, C, OC, mm.ACT_SILU, mm.BF16))
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1]) and torch.equal(res, want[0])
    assert (room[:, :shift] == 3).all() and (room[:, shift + T * OC:] == 3).all()


@pytest.mark.parametrize("path", ["32", "64"])
@pytest.mark.parametrize("size", [(2000, 64, 40), (1300, 36, 20), (40, 68, 3000), (130, 1028, 68), (3, 4000, 100), (700, 500, 36)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fp32_sums_shared_by_blocks(monkeypatch, size, path):
    """Few tiles and long sums, of either product: forward, both gradients, dbias."""
    monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)
    x = inputs(*size, "f32", 51)
    first = check_forward(x, "gelu", "f32")
    assert all(torch.equal(a, b) for a, b in zip(forward(x, "gelu", "f32"), first))
    y = gradient_inputs(*size, "f32", "silu", 52)
    first = check_run(y, "silu", "f32")
    for got in (run(y, "silu", "f32"), run(y, "silu", "f32", in_place=True)):
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("T", [33, 65, 119, 256, 509])
@pytest.mark.parametrize("size", [(8, 8), (1720, 536), (3000, 72), (264, 1000)], ids=lambda s: "x".join(map(str, s)))
def test_forward_of_prompts(T, size):
    """Few tiles: K shared by the warps of a block, tokens in several rows of blocks."""
    x = inputs(T, *size, "bf16", 61)
    first = check_forward(x, "gelu", "bf16")
    for got in (forward(x, "gelu", "bf16"), forward(x, "gelu", "bf16", pre=False, in_place=True)):
        assert torch.equal(got[0], first[0])
