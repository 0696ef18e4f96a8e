"""Host side of the 8-bit linear layer, without a GPU."""
import pytest

import linear_layer_gemms_gb300 as mm


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_layer_gemms_gb300 import _build

    _build.build()
    mm.load()


def test_selftest_of_no_kernel_is_refused():
    assert mm.mmbwd_q8_selftest_wait_timeout(2, 1000) == mm.ERR_SHAPE
    assert mm.mmbwd_q8_selftest_wait_timeout(-1, 1000) == mm.ERR_SHAPE
