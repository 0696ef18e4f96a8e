"""How near the fp32 epilogues come to 64 bits where the bounds of a whole product are too
wide to tell: the activations' derivatives by themselves, and reductions of several
hundred thousand values."""
import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm
from test_gpu_epilogue import ACT, lib, no_failed_wait, ok  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def narrow_slope_bound(x, act):
    """What act'(x) = s + x s c v' may lose, s = sigma(v) and c = 1 - s = e^-v s. v is off by
    six steps of itself (U: half a step) and the exponential by eight (ex2.approx's 2^-22 and
    expf's 2 are below), E = (6 |v| + 8) U relatively, which changes s by c E and c by s E; the
    sum and the reciprocal or division behind s cost at most four more, the products of the second term
    eight, the last addition and product two of the result. No term is a difference of near
    values, so the bound is some 1e-6 at most, where 1 - s as a subtraction costs 2e-6 and
    more of GELU's derivative from x = 5 on."""
    if act in ("none", "relu"):
        return 0 * x
    v = ref.logistic_argument(x, act)
    dv = ref.act_slope(x, "none") if act == "silu" else 2 * (2 / torch.pi) ** 0.5 * (1 + 3 * 0.044715 * x ** 2)
    s, c = torch.sigmoid(v), torch.sigmoid(-v)
    e = (6 * v.abs() + 8) * ref.U
    slope = s + x * s * c * dv
    return s * (c * e + 4 * ref.U) + x.abs() * s * c * dv * (e + 12 * ref.U) + 2 * ref.U * slope.abs() + 2.0 ** -110


@pytest.mark.parametrize("path", ["32", "64", "spans", "alone"])
@pytest.mark.parametrize("act", ref.ACTS)
def test_fp32_derivatives(monkeypatch, act, path):
    """dout . weight is exactly 1 everywhere, so that dpre is the derivative."""
    T, C, OC = 300, 260, 8
    far = 9.9 if act == "gelu" else 80.0
    pre = torch.cat([torch.linspace(-far, far, T * C // 2, dtype=torch.float64), torch.linspace(-7, 7, T * C - T * C // 2, dtype=torch.float64)])
    pre = ref.rounded(pre.cuda().view(T, C), "f32")
    dpre = torch.full((T, C), float("nan"), device="cuda")
    if path == "alone":
        ok(mm.mmbwd_act_backward(dpre, torch.ones_like(dpre), pre.float(), T * C, ACT[act], mm.F32))
    else:
        monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)
        dout, weight = torch.zeros(T, OC, device="cuda"), torch.zeros(OC, C, device="cuda")
        dout[:, 0] = weight[0] = 1.0
        ok(mm.mmbwd_run_act(dpre, torch.zeros_like(weight), None, dout, torch.zeros_like(dpre), weight, pre.float(), None, 0, 1, T, C,
                            OC, ACT[act], mm.F32))
    ref.check(dpre, ref.act_slope(pre, act), narrow_slope_bound(pre, act), "derivative")


def long_sum_bound(length, path):
    """Relative error, in the 2-norm, of sums of `length` products of random operands, whose partial
    sums grow with the square root of what is in them, so that roundings of U of each on a
    chain of n additions are U sqrt(n / 2) of the last sum. Fused multiply-adds: chains of an
    eighth of the length at most, one rounding each, and a few to join them. Three tf32 products:
    32 U of each product (lo lo' and the bits of lo that are not read), the sixteen steps of
    a span that are cut, by 2 U each at most, 2 U sum sqrt(j / 16) = 23 U, and two
    roundings a span of 128 on the running sum."""
    fma = (length / 16) ** 0.5 + 8
    spans = 32 + 23 + (length / 128) ** 0.5
    return {"32": fma, "64": fma, "spans": spans, None: max(fma, spans)}[path] * ref.U


@pytest.mark.parametrize("path", [None, "32", "64", "spans"])
def test_fp32_sums_of_many_values(monkeypatch, path):
    """Reductions of 262,180 and 300,005 values: the forward's, dweight's and dbias'."""
    if path:
        monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)

    def near(got, want, length, path):
        error = ((got.double() - want).norm() / want.norm()).item()
        assert error <= long_sum_bound(length, path), (error, long_sum_bound(length, path))

    T, K, OC = 130, 262_180, 68
    x, w = ref.rounded(ref.normal(1, T, K), "f32"), ref.rounded(ref.normal(2, OC, K), "f32")
    out = torch.empty(T, OC, device="cuda")
    ok(mm.mmbwd_forward_act(out, None, x.float(), w.float(), None, None, 1, T, K, OC, mm.ACT_NONE, mm.F32))
    near(out, x @ w.t(), K, path)
    T, C, OC = 300_005, 68, 36
    dout, inp, w = ref.rounded(ref.normal(3, T, OC), "f32"), ref.rounded(ref.normal(4, T, C), "f32"), ref.rounded(ref.normal(5, OC, C), "f32")
    dpre, dweight, dbias = torch.empty(T, C, device="cuda"), torch.zeros(OC, C, device="cuda"), torch.empty(OC, device="cuda")
    ok(mm.mmbwd_run_act(dpre, dweight, dbias, dout.float(), inp.float(), w.float(), None, None, 0, 1, T, C, OC, mm.ACT_NONE, mm.F32))
    near(dweight, dout.t() @ inp, T, path)
    near(dbias, dout.sum(0), T, "32")  # plain fp32 sums, in chains of an eighth at most
