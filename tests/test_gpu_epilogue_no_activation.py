"""Gradients of a layer without an activation: mmbwd_run_act and mmbwd_act_backward with
ACT_NONE have no use for the activation's argument."""
import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm
from test_gpu_epilogue import DT, dev, gradient_inputs, lib, no_failed_wait, ok, workspace  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
NAN = float("nan")
PATHS = [("bf16", None), ("f32", "32"), ("f32", "64"), ("f32", "spans")]


def call(x, dtype, pre):
    T, C = x["inp"].shape
    OC = x["weight"].shape[0]
    d = {k: dev(v, dtype) for k, v in x.items()}
    room = torch.full((T * C + 512,), 3.0, device="cuda", dtype=ref.TDT[dtype])
    dpre, dbias = room[256:256 + T * C].view(T, C), torch.full((OC,), NAN, device="cuda", dtype=ref.TDT[dtype])
    dpre.fill_(NAN)
    ws, n = workspace(T, C, OC, dtype)
    ok(mm.mmbwd_run_act(dpre, d["dweight"], dbias, d["dout"], d["inp"], d["weight"], pre, ws, n, 1, T, C, OC, mm.ACT_NONE, DT[dtype]))
    assert (room[:256] == 3).all() and (room[256 + T * C:] == 3).all()
    return dpre, d["dweight"], dbias


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("size", [(1, 8, 8), (63, 264, 136), (300, 520, 72), (129, 2056, 264), (2600, 1608, 1000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gradients_without_an_argument(monkeypatch, size, dtype, path):
    if path:
        monkeypatch.setenv("MMBWD_ACT_F32_PATH", path)
    x = gradient_inputs(*size, dtype, "none", 5)
    x["pre"] = torch.full_like(x["inp"], NAN)  # what is passed as the argument has no bearing
    first = call(x, dtype, None)
    want = ref.run_act(x["dout"], x["inp"], x["weight"], 0 * x["inp"], x["dweight"], "none", dtype)
    for name, g, w in zip(("dpre", "dweight", "dbias"), first, want):
        ref.check(g, *w, name)
    for pre in (dev(x["pre"], dtype), None):
        assert all(torch.equal(a, b) for a, b in zip(call(x, dtype, pre), first))


@pytest.mark.parametrize("splits", ["1", "3"])
def test_split_reductions(monkeypatch, splits):
    monkeypatch.setenv("MMBWD_SPLITK", splits)
    x = gradient_inputs(1500, 904, 520, "bf16", "none", 6)
    got = call(x, "bf16", None)
    for name, g, w in zip(("dpre", "dweight", "dbias"), got, ref.run_act(x["dout"], x["inp"], x["weight"], x["pre"], x["dweight"], "none", "bf16")):
        ref.check(g, *w, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alone_is_a_copy(dtype):
    for n in (1, 7, 8, 4095, 100_003):
        d = dev(ref.rounded(ref.normal(8, n), dtype), dtype)
        out = torch.full((n + 64,), 7.0, device="cuda", dtype=ref.TDT[dtype])
        ok(mm.mmbwd_act_backward(out, d, None, n, mm.ACT_NONE, DT[dtype]))
        assert torch.equal(out[:n], d) and (out[n:] == 7).all()
        kept = d.clone()
        ok(mm.mmbwd_act_backward(d, d, None, n, mm.ACT_NONE, DT[dtype]))
        assert torch.equal(d, kept)
