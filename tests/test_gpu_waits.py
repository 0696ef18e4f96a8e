"""The bounded waits of the bf16 / fp32 tensor-core kernel do not count the time of
the launch before their own: a launch that lets the next one begin early and
stays ten times as long as a wait may last."""
import pytest

import linear_layer_gemms_gb300 as mm
import oracle
import synth
from gpu_helpers import assert_close, to_dev, to_host

pytestmark = pytest.mark.gpu
LIMIT, HOLD = "5000000", 50_000_000  # ns
B, T, C, OC = 2, 300, 264, 392


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()


def held(monkeypatch, call):
    """`call` on a stream of its own behind the held launch."""
    import torch

    monkeypatch.setenv("MMBWD_WAIT_TIMEOUT_NS", LIMIT)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        assert mm.mmbwd_debug_hold_stream(HOLD) == mm.OK
        assert call() == mm.OK
    torch.cuda.synchronize()
    assert mm.mmbwd_device_status()[0] == mm.OK


@pytest.mark.parametrize("splits", ["1", "2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(monkeypatch, dtype, splits):
    monkeypatch.setenv("MMBWD_SPLITK", splits)
    code = mm.BF16 if dtype == "bf16" else mm.F32
    x = synth.make_inputs(synth.Layer("case", B, T, C, OC, dtype, True, init_std=0.01, dout_std=1.0, layer=0), seed=0)
    g = {k: to_dev(v, dtype) for k, v in x.items()}
    warm = {k: to_dev(v, dtype) for k, v in x.items()}  # the workspace grows outside the held call
    names = ("dinp", "dweight", "dbias", "dout", "inp", "weight")
    assert mm.mmbwd_run(*(warm[n] for n in names), B, T, C, OC, code) == mm.OK
    held(monkeypatch, lambda: mm.mmbwd_run(*(g[n] for n in names), B, T, C, OC, code))
    want = oracle.get("omp").matmul_backward(x["dout"], x["inp"], x["weight"], dtype, x["dinp"], x["dweight"])
    for name, r in zip(("dinp", "dweight", "dbias"), want):
        assert_close(to_host(g[name], dtype), r, dtype, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(monkeypatch, dtype):
    import torch

    code = mm.BF16 if dtype == "bf16" else mm.F32
    x = {"inp": synth.normal((B * T, C), dtype, 0, 61, 0.0, 1.0), "weight": synth.normal((OC, C), dtype, 0, 62, 0.0, 0.02),
         "bias": synth.normal((OC,), dtype, 0, 63, 0.0, 0.02)}
    g = {k: to_dev(v, dtype) for k, v in x.items()}
    out = torch.full((B * T, OC), float("nan"), dtype=g["inp"].dtype, device="cuda")
    held(monkeypatch, lambda: mm.mmbwd_forward(out, g["inp"], g["weight"], g["bias"], B, T, C, OC, code))
    v = {k: synth.to_f64(a, dtype) for k, a in x.items()}
    assert_close(to_host(out, dtype), v["inp"] @ v["weight"].T + v["bias"], dtype, "out")
