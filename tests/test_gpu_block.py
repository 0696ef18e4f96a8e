"""The operators around the linear layer together, as a training step and a decoding step
use them: norm around the residual, a two-layer MLP with GELU and the residual in its
epilogues, back through all of it, and the gradients clipped by their norm."""
import threading

import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm

pytestmark = pytest.mark.gpu
DT = {"bf16": mm.BF16, "f32": mm.F32}
SCALE = 0.5  # exact in every type
NAN = float("nan")
LEAVES = ("x", "branch", "gate", "weight", "bias", "w1", "b1", "w2", "b2")
STATS = ("mean_post", "rstd_post", "mean", "rstd")


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


def values(T, C, H, dtype, seed=0):
    n = lambda k, *s, std=1.0: ref.rounded(ref.normal(seed + k, *s, std=std), dtype)  # noqa: E731
    return dict(x=n(1, T, C), branch=n(2, T, C), gate=n(3, C), weight=ref.rounded(n(4, C, std=0.1) + 1, dtype), bias=n(5, C, std=0.1),
                w1=n(6, H, C, std=C ** -0.5), b1=n(7, H, std=0.1), w2=n(8, C, H, std=H ** -0.5), b2=n(9, C, std=0.1), dy=n(10, T, C))


class Step:
    """The buffers of a step, and its calls: the norm after the branch is RMS with a gate,
    the norm before the MLP a LayerNorm."""

    def __init__(self, v, dtype, weight_post):
        self.library_ws = True  # the first layer's gradients from mmbwd_run, in the library's own workspace
        self.T, self.C = v["x"].shape
        self.H, self.dtype = v["w1"].shape[0], dtype
        self.v = {k: t.to(ref.TDT[dtype]) for k, t in v.items()}
        self.v["weight_post"] = weight_post.to(ref.TDT[dtype])
        T, C, H = self.T, self.C, self.H
        e = lambda *s: torch.full(s, NAN, device="cuda", dtype=ref.TDT[dtype])  # noqa: E731
        self.r, self.h, self.pre, self.a, self.y = e(T, C), e(T, C), e(T, H), e(T, H), e(T, C)
        self.s = [None] + [torch.full((T,), NAN, device="cuda") for _ in STATS[1:]]
        self.dpre, self.dh, self.dx, self.dbranch = e(T, H), e(T, C), e(T, C), e(T, C)
        self.names = ("gate", "weight_post", "weight", "bias", "w1", "b1", "w2", "b2")
        self.grads = {k: torch.zeros_like(self.v[k]) for k in self.names}
        self.norm = torch.full((1,), NAN, device="cuda")
        room = lambda n: torch.full((max(n, 1),), 0xFF, device="cuda", dtype=torch.uint8)  # noqa: E731
        self.n_run = mm.mmbwd_run_act_workspace_bytes(1, T, H, C, DT[dtype])
        self.n_res = mm.lnbwd_residual_backward_workspace_bytes(1, T, C, DT[dtype])
        self.n_clip = mm.mmbwd_grad_workspace_bytes(len(self.grads))
        self.n_first = mm.mmbwd_run_act_workspace_bytes(1, T, C, H, DT[dtype])
        self.ws = room(self.n_run), room(self.n_res), room(self.n_clip), room(self.n_first)
        self.unclipped = {k: torch.zeros_like(t) for k, t in self.grads.items()}
        self.list = mm.grad_list([(self.unclipped[k], g, g.numel(), DT[dtype]) for k, g in self.grads.items()])

    def forward(self, stream=None):
        v, T, C, H, d = self.v, self.T, self.C, self.H, DT[self.dtype]
        ok(mm.lnbwd_residual_forward(self.h, self.r, *self.s, v["x"], v["branch"], v["gate"], v["weight_post"], None, v["weight"], v["bias"],
                                     1, T, C, SCALE, ref.EPS, mm.NORM_RMS, mm.NORM_LAYER, d, stream=stream))
        ok(mm.mmbwd_forward_act(self.a, self.pre, self.h, v["w1"], v["b1"], None, 1, T, C, H, mm.ACT_GELU, d, stream=stream))
        ok(mm.mmbwd_forward_act(self.y, None, self.a, v["w2"], v["b2"], self.r, 1, T, H, C, mm.ACT_NONE, d, stream=stream))

    def backward(self, max_norm, stream=None):
        v, g, T, C, H, d = self.v, self.unclipped, self.T, self.C, self.H, DT[self.dtype]
        w_run, w_res, w_clip, w_first = self.ws
        ok(mm.mmbwd_run_act(self.dpre, g["w2"], g["b2"], v["dy"], self.a, v["w2"], self.pre, w_run if self.n_run else None, self.n_run, 1, T,
                            H, C, mm.ACT_GELU, d, stream=stream))
        if self.library_ws:
            ok(mm.mmbwd_run(self.dh, g["w1"], g["b1"], self.dpre, self.h, v["w1"], 1, T, C, H, d, stream=stream))
        else:
            ok(mm.mmbwd_run_act(self.dh, g["w1"], g["b1"], self.dpre, self.h, v["w1"], self.h, w_first if self.n_first else None,
                                self.n_first, 1, T, C, H, mm.ACT_NONE, d, stream=stream))
        ok(mm.lnbwd_residual_backward(self.dx, self.dbranch, g["gate"], g["weight_post"], None, g["weight"], g["bias"], self.dh, v["dy"],
                                      self.r, v["branch"], v["gate"], v["weight_post"], None, v["weight"], *self.s, w_res, self.n_res, 1,
                                      T, C, SCALE, mm.NORM_RMS, mm.NORM_LAYER, d, stream=stream))
        ok(mm.mmbwd_grad_clip(self.norm, self.list, max_norm, w_clip, self.n_clip, stream=stream))

    def clear(self):
        self.dh.zero_()
        for t in self.unclipped.values():
            t.zero_()

    def results(self):
        return [t.clone() for t in (self.r, self.h, self.pre, self.a, self.y, self.dpre, self.dh, self.dx, self.dbranch, self.norm,
                                    *self.unclipped.values(), *self.grads.values())]


def make(T, C, H, dtype, seed=0):
    v = values(T, C, H, dtype, seed)
    return v, Step(v, dtype, ref.rounded(ref.normal(seed + 11, C, std=0.1) + 1, dtype))


def run(step, max_norm):
    step.clear()
    torch.cuda.synchronize()
    step.forward()
    step.backward(max_norm)
    torch.cuda.synchronize()


SIZES = [(1, 64, 256), (37, 264, 1056), (300, 768, 1000), (129, 1600, 6400)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_each_operator_of_a_step(size, dtype):
    """Every operator from what the ones before it stored, with its own bound."""
    v, p = make(*size, dtype)
    run(p, 1e-2)
    w = {k: t.double() for k, t in p.v.items()}
    want = ref.residual_forward(w["x"], w["branch"], w["gate"], w["weight_post"], None, w["weight"], w["bias"], SCALE, "rms", "layer", dtype)
    for k, t in dict(residual_out=p.r, out=p.h, rstd_post=p.s[1], mean=p.s[2], rstd=p.s[3]).items():
        ref.check(t, *want[k], k)
    out, pre = ref.forward_act(p.h.double(), w["w1"], w["b1"], None, "gelu", dtype)
    ref.check(p.a, *out, "a")
    ref.check(p.pre, *pre, "pre")
    ref.check(p.y, *ref.forward_act(p.a.double(), w["w2"], w["b2"], p.r.double(), "none", dtype)[0], "y")
    for t, want, k in zip((p.dpre, p.unclipped["w2"], p.unclipped["b2"]),
                          ref.run_act(w["dy"], p.a.double(), w["w2"], p.pre.double(), torch.zeros_like(w["w2"]), "gelu", dtype),
                          ("dpre", "w2", "b2")):
        ref.check(t, *want, k)
    if dtype == "bf16":  # (mmbwd_run's fp32 products have a bound of their own, and the test below)
        for t, want, k in zip((p.dh, p.unclipped["w1"], p.unclipped["b1"]),
                              ref.run_act(p.dpre.double(), p.h.double(), w["w1"], p.h.double(), torch.zeros_like(w["w1"]), "none", dtype),
                              ("dh", "w1", "b1")):
            ref.check(t, *want, k)
    old = dict(dgate=0 * w["gate"], dweight_post=0 * w["gate"], dweight=0 * w["gate"], dbias=0 * w["gate"])
    want = ref.residual_backward(p.dh.double(), w["dy"], p.r.double(), w["branch"], w["gate"], w["weight_post"], None, w["weight"],
                                 [None] + [t.double() for t in p.s[1:]], old, SCALE, "rms", "layer", dtype)
    got = dict(dx=p.dx, dbranch=p.dbranch, dgate=p.unclipped["gate"], dweight_post=p.unclipped["weight_post"],
               dweight=p.unclipped["weight"], dbias=p.unclipped["bias"])
    for k, t in got.items():
        ref.check(t, *want[k], k)
    # the norm: 64 roundings of fp32 in a thread's sum of squares, half of that in the root
    norm = sum(t.double().square().sum() for t in p.unclipped.values()).sqrt().item()
    assert abs(p.norm.item() - norm) <= 40 * ref.U * norm
    coef = min(1.0, 1e-2 / (norm + 1e-6))
    for k, g in p.grads.items():
        t = p.unclipped[k].double() * coef
        ref.check(g, t, ref.stored(48 * ref.U * t.abs(), t, dtype), "clipped " + k)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_gradients_of_a_step(size):
    """fp32 against 64-bit automatic differentiation of the definitions. On the longest path
    are 12 products, norms and sums, each off by at most 1e-6 in the 2-norm, but for mmbwd_run's
    product (1.2e-5 at 1600 values, growing with their number; 6400 here: 5e-5). An earlier
    error grows at most threefold (the weights' columns have norms near 1, GELU's slope is at most
    1.13, each rstd near 1, and the residual keeps what is added to it):
    3 * (5e-5 + 11e-6) < 3e-4."""
    v, p = make(*size, "f32", 100)
    run(p, 1e30)
    leaf = {k: v[k].clone().requires_grad_() for k in LEAVES}
    wp = p.v["weight_post"].double().requires_grad_()
    b, x = leaf["branch"], leaf["x"]
    z = b / (b.square().mean(1, keepdim=True) + ref.EPS).sqrt() * wp
    r = x + SCALE * leaf["gate"] * z
    h = torch.nn.functional.layer_norm(r, (p.C,), leaf["weight"], leaf["bias"], ref.EPS)
    a = torch.nn.functional.gelu(h @ leaf["w1"].t() + leaf["b1"], approximate="tanh")
    y = r + a @ leaf["w2"].t() + leaf["b2"]
    y.backward(v["dy"])
    assert (p.y - y).norm() <= 1e-5 * y.norm()
    got = dict(p.unclipped, x=p.dx, branch=p.dbranch)
    for k in LEAVES + ("weight_post",):
        want = wp.grad if k == "weight_post" else leaf[k].grad
        assert (got[k].double() - want).norm() <= 3e-4 * want.norm(), k
    for k, g in p.grads.items():  # under the limit: as they are
        assert torch.equal(g, p.unclipped[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_step_in_a_graph(dtype):
    v, p = make(300, 264, 1056, dtype)
    run(p, 0.5)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    p.clear()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        p.clear()
        p.forward(s.cuda_stream)
        p.backward(0.5, s.cuda_stream)
    u = values(300, 264, 1056, dtype, 500)
    for k, t in u.items():
        p.v[k].copy_(t)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    got = p.results()
    run(p, 0.5)
    for a, b in zip(got, p.results()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_step_needs_only_the_weights_gradients_cleared(dtype):
    """Both layers' gradients by mmbwd_run_act, as the documented sequence has them: whatever
    the last step left in the other buffers has no bearing."""
    v, p = make(200, 264, 1056, dtype, 40)
    p.library_ws = False
    run(p, 0.5)
    want = p.results()
    for k, t in p.unclipped.items():
        t.fill_(NAN if k in ("b1", "b2") else 0.0)
    for t in (p.dh, p.dpre, p.dx, p.dbranch, p.norm, *p.grads.values(), p.r, p.h, p.pre, p.a, p.y):
        t.fill_(NAN)
    p.forward()
    p.backward(0.5)
    torch.cuda.synchronize()
    for a, b in zip(p.results(), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decoding_tokens_one_at_a_time(dtype):
    """The forward of a token alone has the same result whatever the others are: each row of
    a batch within the two calls' bounds of the row by itself."""
    v, p = make(40, 264, 1056, dtype)
    p.forward()
    want = {k: getattr(p, k).clone() for k in ("r", "h")}
    torch.cuda.synchronize()
    for t in (0, 17, 39):
        w = {k: (x[t:t + 1] if k in ("x", "branch", "dy") else x) for k, x in v.items()}
        one = Step(w, dtype, p.v["weight_post"].double())
        one.forward()
        d = {k: x.double() for k, x in one.v.items()}
        out, pre = ref.forward_act(one.h.double(), d["w1"], d["b1"], None, "gelu", dtype)
        ref.check(one.a, *out, "a")
        ref.check(one.y, *ref.forward_act(one.a.double(), d["w2"], d["b2"], one.r.double(), "none", dtype)[0], "y")
        res = ref.residual_forward(d["x"], d["branch"], d["gate"], d["weight_post"], None, d["weight"], d["bias"], SCALE, "rms", "layer", dtype)
        for k, name in (("r", "residual_out"), ("h", "out")):
            ref.check(getattr(one, k), *res[name], k)
            ref.check(want[k][t:t + 1], *res[name], k)


def test_steps_of_several_threads():
    """Threads that call at once, each on a stream of its own with its own workspaces."""
    steps = [make(200, 264, 1056, "bf16", 1000 * i)[1] for i in range(4)]
    want = []
    for p in steps:
        p.library_ws = False
        run(p, 0.5)
        want.append(p.results())
    streams = [torch.cuda.Stream() for _ in steps]
    errors = []

    def work(p, s):
        try:
            torch.cuda.set_device(0)
            for _ in range(10):
                with torch.cuda.stream(s):
                    p.clear()
                p.forward(s.cuda_stream)
                p.backward(0.5, s.cuda_stream)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(steps, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for p, w in zip(steps, want):
        for a, b in zip(p.results(), w):
            assert torch.equal(a, b)
