"""Refusals and sizes of the operators around the linear layer (activation and residual
epilogues, norms around a block, gradient norm and clipping), without a GPU; and the
reference that their GPU tests use, against differentiation."""
import ctypes

import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_layer_gemms_gb300 import _build

    _build.build()
    mm.load()


A = 1 << 24  # fake, aligned addresses: validation fails before any use


def forward(**kw):
    a = dict(out=A, pre=2 * A, inp=3 * A, weight=4 * A, bias=5 * A, residual=6 * A, B=2, T=8, C=64, OC=32, act=mm.ACT_GELU,
             dtype=mm.BF16, stream=0)
    a.update(kw)
    return mm.mmbwd_forward_act(**a)


def test_forward_act_refusals():
    assert forward(dtype=2) == mm.ERR_DTYPE
    assert forward(act=4) == mm.ERR_SHAPE
    assert forward(act=-1) == mm.ERR_SHAPE
    assert forward(T=-1) == mm.ERR_SHAPE
    assert forward(B=1 << 20, T=1 << 20) == mm.ERR_SHAPE
    assert forward(OC=(65535 * 128) + 8, C=0, T=0) == mm.ERR_SHAPE
    assert forward(out=None) == mm.ERR_NULL
    assert forward(inp=None) == mm.ERR_NULL
    assert forward(weight=None) == mm.ERR_NULL
    assert forward(C=60) == mm.ERR_ALIGN
    assert forward(OC=36) == mm.ERR_ALIGN
    assert forward(C=62, dtype=mm.F32) == mm.ERR_ALIGN
    assert forward(pre=2 * A + 8) == mm.ERR_ALIGN
    assert forward(residual=6 * A + 2) == mm.ERR_ALIGN
    assert forward(out=3 * A + 64) == mm.ERR_ALIAS
    assert forward(pre=A + 64) == mm.ERR_ALIAS
    assert forward(pre=6 * A) == mm.ERR_ALIAS  # the residual is read after pre is written
    assert forward(residual=A + 64) == mm.ERR_ALIAS  # in place is the same place
    assert forward(bias=2 * A + 16) == mm.ERR_ALIAS


def run(**kw):
    a = dict(dpre=A, dweight=2 * A, dbias=3 * A, dout=4 * A, inp=5 * A, weight=6 * A, pre=7 * A, workspace=8 * A,
             workspace_bytes=1 << 23, B=2, T=8, C=64, OC=32, act=mm.ACT_SILU, dtype=mm.BF16, stream=0)
    a.update(kw)
    return mm.mmbwd_run_act(**a)


def test_run_act_refusals(monkeypatch):
    assert run(dtype=3) == mm.ERR_DTYPE
    assert run(act=9) == mm.ERR_SHAPE
    assert run(C=-8) == mm.ERR_SHAPE
    for name in ("dpre", "dweight", "dout", "inp", "weight", "pre"):
        assert run(**{name: None}) == mm.ERR_NULL, name
    assert run(C=60) == mm.ERR_ALIGN
    assert run(pre=7 * A + 8) == mm.ERR_ALIGN
    assert run(workspace=8 * A + 16) == mm.ERR_ALIGN
    assert run(dpre=5 * A) == mm.ERR_ALIAS  # the activation is read by the other product
    assert run(dpre=7 * A + 64) == mm.ERR_ALIAS
    assert run(dweight=A + 64) == mm.ERR_ALIAS
    assert run(dbias=7 * A) == mm.ERR_ALIAS
    monkeypatch.setenv("MMBWD_SPLITK", "3")
    size = dict(B=1, T=1000, C=264, OC=392)
    need = mm.mmbwd_run_act_workspace_bytes(*size.values(), mm.BF16)
    assert need > 0 and mm.mmbwd_run_act_workspace_bytes(*size.values(), mm.F32) == 0
    assert run(**size, workspace_bytes=need - 1) == mm.ERR_SHAPE
    assert run(**size, workspace=None) == mm.ERR_NULL
    assert run(**size, workspace=4 * A) == mm.ERR_ALIAS
    assert run(**size, dout=8 * A + need - 16) == mm.ERR_ALIAS
    assert mm.mmbwd_run_act_workspace_bytes(-1, 8, 64, 64, mm.BF16) == 0


def alone(**kw):
    a = dict(dpre=A, dout=2 * A, pre=3 * A, n=1001, act=mm.ACT_RELU, dtype=mm.F32, stream=0)
    a.update(kw)
    return mm.mmbwd_act_backward(**a)


def test_act_backward_refusals():
    assert alone(dtype=-1) == mm.ERR_DTYPE
    assert alone(act=7) == mm.ERR_SHAPE
    assert alone(n=-1) == mm.ERR_SHAPE
    assert alone(n=1 << 60) == mm.ERR_SHAPE
    assert alone(dout=None) == mm.ERR_NULL
    assert alone(pre=3 * A + 4) == mm.ERR_ALIGN
    assert alone(dpre=2 * A + 16) == mm.ERR_ALIAS


def test_no_activation_has_no_argument():
    """ACT_NONE does not look at pre: none at all, unaligned, inside an output."""
    for pre in (None, 7 * A + 8, 2 * A, A + 64):
        refused = (mm.ERR_NULL, mm.ERR_ALIGN, mm.ERR_ALIAS)
        assert run(pre=pre) in refused and run(pre=pre, act=mm.ACT_NONE) not in refused
        assert alone(pre=pre, act=mm.ACT_NONE) not in refused
    assert alone(pre=None) == mm.ERR_NULL


def norms(**kw):
    a = dict(out=A, residual_out=2 * A, mean_post=3 * A, rstd_post=4 * A, mean=5 * A, rstd=6 * A, x=7 * A, branch=8 * A,
             gate=9 * A, weight_post=10 * A, bias_post=11 * A, weight=12 * A, bias=13 * A, B=2, T=8, C=64, scale=0.5,
             eps=1e-5, post=mm.NORM_LAYER, norm=mm.NORM_LAYER, dtype=mm.BF16, stream=0)
    a.update(kw)
    return mm.lnbwd_residual_forward(**a)


def test_residual_forward_refusals():
    assert norms(dtype=2) == mm.ERR_DTYPE
    assert norms(post=3) == mm.ERR_SHAPE
    assert norms(norm=-1) == mm.ERR_SHAPE
    assert norms(C=mm.RESIDUAL_MAX_C + 8) == mm.ERR_SHAPE
    assert norms(scale=float("inf")) == mm.ERR_SHAPE
    assert norms(scale=float("nan")) == mm.ERR_SHAPE
    assert norms(eps=-1.0) == mm.ERR_SHAPE
    assert norms(eps=float("nan")) == mm.ERR_SHAPE
    for name in ("out", "residual_out", "x", "branch", "weight_post", "weight"):
        assert norms(**{name: None}) == mm.ERR_NULL, name
    assert norms(C=60) == mm.ERR_ALIGN
    assert norms(branch=8 * A + 8) == mm.ERR_ALIGN
    assert norms(mean=5 * A + 2) == mm.ERR_ALIGN
    assert norms(residual_out=8 * A) == mm.ERR_ALIAS
    assert norms(residual_out=7 * A + 128) == mm.ERR_ALIAS
    assert norms(out=2 * A) == mm.ERR_ALIAS
    assert norms(out=7 * A) == mm.ERR_ALIAS
    assert norms(rstd=5 * A + 32) == mm.ERR_ALIAS
    assert norms(mean_post=A + 64) == mm.ERR_ALIAS
    assert norms(rstd_post=12 * A) == mm.ERR_ALIAS


def grads(**kw):
    a = dict(dx=A, dbranch=2 * A, dgate=3 * A, dweight_post=4 * A, dbias_post=5 * A, dweight=6 * A, dbias=7 * A, dout=8 * A,
             dresidual=9 * A, residual=10 * A, branch=11 * A, gate=12 * A, weight_post=13 * A, bias_post=14 * A, weight=15 * A,
             mean_post=16 * A, rstd_post=17 * A, mean=18 * A, rstd=19 * A, workspace=20 * A, workspace_bytes=1 << 23, B=2, T=8,
             C=64, scale=0.5, post=mm.NORM_LAYER, norm=mm.NORM_LAYER, dtype=mm.BF16, stream=0)
    a.update(kw)
    return mm.lnbwd_residual_backward(**a)


def test_residual_backward_refusals():
    assert grads(dtype=2) == mm.ERR_DTYPE
    assert grads(post=5) == mm.ERR_SHAPE
    assert grads(C=mm.RESIDUAL_MAX_C + 8) == mm.ERR_SHAPE
    assert grads(scale=float("-inf")) == mm.ERR_SHAPE
    for name in ("dx", "dout", "residual", "branch", "weight_post", "weight", "mean_post", "rstd_post", "mean", "rstd",
                 "workspace"):
        assert grads(**{name: None}) == mm.ERR_NULL, name
    assert grads(norm=mm.NORM_NONE, dresidual=None) == mm.ERR_NULL
    assert grads(C=60) == mm.ERR_ALIGN
    assert grads(dgate=3 * A + 8) == mm.ERR_ALIGN
    assert grads(rstd=19 * A + 1) == mm.ERR_ALIGN
    assert grads(workspace=20 * A + 16) == mm.ERR_ALIGN
    need = mm.lnbwd_residual_backward_workspace_bytes(2, 8, 64, mm.BF16)
    assert need > 0 and grads(workspace_bytes=need - 1) == mm.ERR_SHAPE
    assert mm.lnbwd_residual_backward_workspace_bytes(2, 0, 64, mm.BF16) == 0
    assert mm.lnbwd_residual_backward_workspace_bytes(2, 8, 60, mm.BF16) == 0
    assert mm.lnbwd_residual_backward_workspace_bytes(2, -8, 64, mm.BF16) == 0
    assert grads(dx=9 * A + 64) == mm.ERR_ALIAS
    assert grads(dx=8 * A) == mm.ERR_ALIAS
    assert grads(dbranch=A) == mm.ERR_ALIAS
    assert grads(dbranch=11 * A) == mm.ERR_ALIAS
    assert grads(dweight=6 * A, dbias=6 * A + 64) == mm.ERR_ALIAS
    assert grads(mean=20 * A) == mm.ERR_ALIAS


def tensors(*rows):
    return mm.grad_list(list(rows))


def clip(rows, norm=A, max_norm=1.0, workspace=2 * A, workspace_bytes=None, n=None):
    n = len(rows) if n is None else n
    size = mm.mmbwd_grad_workspace_bytes(n) if workspace_bytes is None else workspace_bytes
    return mm.load().mmbwd_grad_clip(norm, tensors(*rows), n, max_norm, workspace, size, 0)


def test_grad_refusals():
    good = (3 * A, None, 100, mm.F32)
    assert clip([good], n=-1, workspace_bytes=1 << 20) == mm.ERR_SHAPE
    assert clip([good], max_norm=-1.0) == mm.ERR_SHAPE
    assert clip([good], max_norm=float("nan")) == mm.ERR_SHAPE
    assert clip([good], max_norm=float("inf")) == mm.ERR_SHAPE
    assert clip([(3 * A, None, -1, mm.F32)]) == mm.ERR_SHAPE
    assert clip([(3 * A, None, 1 << 60, mm.F32)]) == mm.ERR_SHAPE
    assert clip([good], workspace_bytes=8) == mm.ERR_SHAPE
    assert clip([(3 * A, None, 5, 2)]) == mm.ERR_DTYPE
    assert clip([good], norm=None) == mm.ERR_NULL
    assert clip([good], workspace=None) == mm.ERR_NULL
    assert clip([(None, None, 5, mm.F32)]) == mm.ERR_NULL
    assert clip([good], norm=A + 2) == mm.ERR_ALIGN
    assert clip([good], workspace=2 * A + 64) == mm.ERR_ALIGN
    assert clip([(3 * A + 2, None, 5, mm.F32)]) == mm.ERR_ALIGN
    assert clip([(3 * A, 4 * A + 1, 5, mm.BF16)]) == mm.ERR_ALIGN
    assert clip([good, good]) == mm.ERR_ALIAS  # in place twice
    assert clip([(3 * A, 4 * A, 100, mm.F32), (5 * A, 3 * A + 396, 100, mm.F32)]) == mm.ERR_ALIAS
    assert clip([(3 * A, 3 * A + 4, 100, mm.F32)]) == mm.ERR_ALIAS
    assert clip([(2 * A + 128, None, 100, mm.F32)]) == mm.ERR_ALIAS
    assert clip([(A - 8, None, 100, mm.F32)]) == mm.ERR_ALIAS
    lib = mm.load()
    assert lib.mmbwd_grad_norm(A, None, 1, 2 * A, 1 << 20, 0) == mm.ERR_NULL
    assert lib.mmbwd_grad_scale(tensors(good), 1, None, 1.0, 0) == mm.ERR_NULL
    assert lib.mmbwd_grad_scale(tensors((A, None, 5, mm.F32)), 1, A, 1.0, 0) == mm.ERR_ALIAS
    assert mm.mmbwd_grad_workspace_bytes(-1) == 0
    assert mm.mmbwd_grad_workspace_bytes(0) > 0
    assert mm.mmbwd_grad_workspace_bytes(1025) == 2 * mm.mmbwd_grad_workspace_bytes(1024)
    assert ctypes.sizeof(mm.Grad) == 32


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_a_gpu_fail_cleanly():
    fails = (mm.ERR_CUDA, mm.ERR_ARCH)
    for call in (forward, run, alone, norms, grads):
        assert call() in fails
    assert forward(residual=A) in fails and run(dpre=7 * A) in fails  # in place is allowed
    assert alone(dout=A) in fails and alone(pre=A) in fails
    assert norms(residual_out=7 * A) in fails and grads(dx=9 * A) in fails
    # what a norm does not have is not looked at
    assert norms(post=mm.NORM_NONE, weight_post=None, bias_post=A, mean_post=A, rstd_post=A + 1) in fails
    assert norms(norm=mm.NORM_NONE, out=None, weight=None, mean=A, rstd=2 * A) in fails
    assert norms(post=mm.NORM_RMS, norm=mm.NORM_RMS, bias_post=A + 1, bias=A + 1, mean=A, mean_post=A) in fails
    assert grads(post=mm.NORM_NONE, dgate=None, branch=None, weight_post=None, rstd_post=None, mean_post=None) in fails
    assert grads(gate=None, dgate=A) in fails
    assert clip([(3 * A, None, 100, mm.F32), (3 * A + 400, None, 100, mm.F32), (None, None, 0, mm.BF16)]) in fails
    lib = mm.load()
    assert lib.mmbwd_grad_norm(A, tensors((3 * A, None, 9, 0), (3 * A, None, 9, 0)), 2, 2 * A, 1 << 20, 0) in fails


# ------------------------------------------------------------------ the reference

@pytest.mark.parametrize("act", ref.ACTS)
def test_reference_activations(act):
    x = torch.linspace(-12, 12, 4001, dtype=torch.float64, requires_grad=True)
    f = torch.nn.functional
    y = {"none": lambda v: v * 1, "gelu": lambda v: f.gelu(v, approximate="tanh"), "silu": f.silu, "relu": f.relu}[act](x)
    torch.testing.assert_close(ref.act_value(x.detach(), act), y.detach(), rtol=1e-9, atol=1e-12)
    keep = x.detach() != 0
    (d,) = torch.autograd.grad(y.sum(), x)
    torch.testing.assert_close(ref.act_slope(x.detach(), act)[keep], d[keep], rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("norm", ref.KINDS)
@pytest.mark.parametrize("post", ref.KINDS)
def test_reference_residual_gradients(post, norm):
    """Against automatic differentiation of the definition."""
    f = torch.nn.functional
    n = lambda k, *s: ref.normal(k, *s, device="cpu")  # noqa: E731
    x, br, gate, wp, bp, w, b = n(1, 5, 16), n(2, 5, 16), n(3, 16), n(4, 16), n(5, 16), n(6, 16), n(7, 16)
    dout, dres, scale = n(8, 5, 16), n(9, 5, 16), 0.7
    leaves = [t.requires_grad_() for t in (x, br, gate, wp, bp, w, b)]

    def apply(v, kind, weight, bias):
        if kind == "layer":
            return f.layer_norm(v, (16,), weight, bias, ref.EPS)
        return f.rms_norm(v, (16,), weight, ref.EPS) if kind == "rms" else v

    r = x + scale * gate * apply(br, post, wp, bp)
    out = apply(r, norm, w, b)
    loss = (r * dres).sum() + ((out * dout).sum() if norm != "none" else 0)
    want = torch.autograd.grad(loss, leaves, allow_unused=True)
    x, br, gate, wp, bp, w, b = (t.detach() for t in leaves)
    fwd = ref.residual_forward(x, br, gate, wp, bp, w, b, scale, post, norm, "f32")
    torch.testing.assert_close(fwd["residual_out"][0], r.detach())
    if norm != "none":
        torch.testing.assert_close(fwd["out"][0], out.detach())
    stats = [fwd[k][0] if k in fwd else None for k in ("mean_post", "rstd_post", "mean", "rstd")]
    names = ["dx", "dbranch", "dgate", "dweight_post", "dbias_post", "dweight", "dbias"]
    old = {k: torch.zeros(16, dtype=torch.float64) for k in names[2:]}
    got = ref.residual_backward(dout, dres, fwd["residual_out"][0], br, gate, wp, bp, w, stats, old, scale, post, norm, "f32")
    for name, g in zip(names, want):
        if g is not None:
            torch.testing.assert_close(got[name][0], g, rtol=1e-9, atol=1e-10, msg=name)
