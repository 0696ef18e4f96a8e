"""The bounded waits of the 8-bit product kernels: one that runs out is reported
and cleared, and none counts the time of the launch before its own."""
import time

import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
from test_gpu_q8 import dev, host, lib, normal, q8, tdt  # noqa: F401

pytestmark = pytest.mark.gpu
SELFTEST = 9  # wait site


def forward_is_right(T, hold_ns=0, C=1032, OC=264):
    import torch

    iq, isc, iv = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, wv = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    out = torch.full((T, OC), float("nan"), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        if hold_ns:
            assert mm.mmbwd_debug_hold_stream(hold_ns) == mm.OK
        assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, T, C, OC, 0, 0, mm.F32) == mm.OK
    torch.cuda.synchronize()
    assert mm.mmbwd_device_status()[0] == mm.OK
    want, tol = ref.product_bound(iv, wv, "f32")
    assert np.all(np.abs(host(out) - want) <= tol)


@pytest.mark.parametrize("kernel", [0, 1], ids=["products", "few tokens"])
def test_a_wait_that_runs_out_is_reported_and_cleared(kernel):
    assert mm.mmbwd_q8_selftest_wait_timeout(kernel, 20_000_000) == mm.OK
    for reset in (False, True):
        assert mm.mmbwd_device_status(reset) == (mm.ERR_DEVICE_TIMEOUT, [0, SELFTEST, 0])
    assert mm.mmbwd_device_status()[0] == mm.OK
    forward_is_right(300 if kernel == 0 else 5)


@pytest.mark.parametrize("kernel", [0, 1], ids=["products", "few tokens"])
def test_the_limit_is_the_one_of_the_environment(monkeypatch, kernel):
    monkeypatch.setenv("MMBWD_WAIT_TIMEOUT_NS", "50000000")
    t0 = time.perf_counter()
    assert mm.mmbwd_q8_selftest_wait_timeout(kernel) == mm.OK
    assert 0.05 <= time.perf_counter() - t0 < 1.5
    assert mm.mmbwd_device_status() == (mm.ERR_DEVICE_TIMEOUT, [0, SELFTEST, 0])


def test_the_selftest_ends_whatever_is_asked_for():
    t0 = time.perf_counter()
    assert mm.mmbwd_q8_selftest_wait_timeout(0, 1 << 62) == mm.OK
    assert time.perf_counter() - t0 < 4
    assert mm.mmbwd_device_status() == (mm.ERR_DEVICE_TIMEOUT, [0, SELFTEST, 0])


@pytest.mark.parametrize("T", [300, 5], ids=["products", "few tokens"])
def test_the_launch_before_does_not_count_against_the_forward(monkeypatch, T):
    """A launch that lets the forward begin early and stays ten times as long as a
    wait may last."""
    monkeypatch.setenv("MMBWD_WAIT_TIMEOUT_NS", "5000000")
    forward_is_right(T, hold_ns=50_000_000)


@pytest.mark.parametrize("splits", ["1,1", "2,3"])
def test_the_launch_before_does_not_count_against_the_backward(monkeypatch, splits):
    import torch

    monkeypatch.setenv("MMBWD_WAIT_TIMEOUT_NS", "5000000")
    monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    T, C, OC = 1400, 392, 1096
    d, inp, w = normal((T, OC), "bf16", 4, 1e-2), normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6, 0.02)
    dq, ds, dv = q8(d, mm.E4M3)
    dqt, dst, dvt = q8(d.T, mm.E4M3)
    iqt, ist, ivt = q8(inp.T, mm.E4M3)
    wqt, wst, wvt = q8(w.T, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    dinp, dw = torch.empty(T, C, device="cuda"), torch.empty(OC, C, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        assert mm.mmbwd_debug_hold_stream(50_000_000) == mm.OK
        assert mm.mmbwd_q8_backward(dinp, dw, dq, ds, dqt, dst, iqt, ist, wqt, wst, ws, n, 1, T, C, OC, 0, 0, 0, mm.F32,
                                    mm.F32, 0) == mm.OK
    torch.cuda.synchronize()
    assert mm.mmbwd_device_status()[0] == mm.OK
    for got, (want, tol) in ((dinp, ref.product_bound(dv, wvt, "f32")), (dw, ref.product_bound(dvt, ivt, "f32"))):
        assert np.all(np.abs(host(got) - want) <= tol)
