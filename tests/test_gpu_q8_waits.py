"""The bounded waits of the 8-bit product kernels: one that runs out is reported
and cleared."""
import time

import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
from test_gpu_q8 import dev, host, lib, normal, q8, tdt  # noqa: F401

pytestmark = pytest.mark.gpu
SELFTEST = 9  # wait site


def forward_is_right(T, C=1032, OC=264):
    import torch

    iq, isc, iv = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, wv = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    out = torch.full((T, OC), float("nan"), device="cuda")
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, T, C, OC, 0, 0, mm.F32) == mm.OK
    torch.cuda.synchronize()
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
