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
