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


def test_shapes_in_rotation_are_planned_once():
    """64 layer shapes, as a model with batches of changing length has: the second
    time round no work split is searched for again, and the sizes are the same."""
    shapes = [(1, 300 + 37 * i, C, OC) for i in range(16)
              for C, OC in ((328, 520), (520, 328), (264, 1032), (1032, 264))]
    before = mm.mmbwd_q8_debug_plan_searches()
    first = [mm.mmbwd_q8_backward_workspace_bytes(*s) for s in shapes]
    made = mm.mmbwd_q8_debug_plan_searches()
    assert made > before
    assert [mm.mmbwd_q8_backward_workspace_bytes(*s) for s in shapes] == first
    assert mm.mmbwd_q8_debug_plan_searches() == made


def test_queries_from_several_threads_agree():
    import threading

    shapes = [(1, 900 + 41 * i, 392, 520) for i in range(24)]
    got = [None] * 4

    def work(k):
        order = shapes if k % 2 else shapes[::-1]
        sizes = {s: mm.mmbwd_q8_backward_workspace_bytes(*s) for s in order * 2}
        got[k] = [sizes[s] for s in shapes]

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got[0] is not None and all(g == got[0] for g in got)


@pytest.mark.parametrize("shape, splits", [((1, 16384, 8192, 2048), "1,2"), ((1, 2048, 8192, 16384), "2,1")],
                         ids=["dweight", "dinp"])
def test_a_forced_split_is_taken_whatever_the_other_products_items(monkeypatch, shape, splits):
    """1024 items of the split product beside 4096 of the other, which comes after it
    in one case and before it in the other."""
    monkeypatch.setenv("MMBWD_Q8_TILE_N", "128,128")
    monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    assert mm.mmbwd_q8_backward_workspace_bytes(*shape) == 1024 * 256 * 128 * 4


def test_many_items_are_not_split_for_the_other_products_length():
    """5120 tiles for 76 pairs: a product with four times the other's reduction has
    enough of them unsplit."""
    assert mm.mmbwd_q8_backward_workspace_bytes(1, 8192, 8192, 32768) == 0


def test_an_override_of_dinp_leaves_dweight_alone(monkeypatch):
    """The size covers dweight alone, which takes the second value: with only dinp
    split, what is needed are dinp's partial tiles (6 tiles of 256 x 256 in 4 splits
    of 16 blocks), not four times dweight's eight tiles."""
    shape = (1, 1400, 256, 2048)
    monkeypatch.setenv("MMBWD_Q8_TILE_N", "256,256")
    monkeypatch.setenv("MMBWD_Q8_SPLITS", "4,1")
    assert mm.mmbwd_q8_backward_workspace_bytes(*shape) == 6 * 4 * 256 * 256 * 4
    monkeypatch.setenv("MMBWD_Q8_SPLITS", "1,4")  # (11 blocks of 128 tokens: 3, 3, 3, 2)
    assert mm.mmbwd_q8_backward_workspace_bytes(*shape) == 8 * 4 * 256 * 256 * 4


@pytest.mark.parametrize("fmt, least", [(mm.E4M3, -124), (mm.E5M2, -117)], ids=["e4m3", "e5m2"])
def test_where_values_times_scales_are_exact(fmt, least):
    """The header's ranges of s: fp32 holds every q 2^s that is under 2^128, bf16 those
    from `least` on and not all below."""
    import numpy as np
    import torch

    import q8_reference as ref

    q = ref.decode(np.arange(256, dtype=np.uint8), fmt)
    q = q[np.isfinite(q)]
    for s in (-127, least, 0, 112, 120):
        v = np.ldexp(q, s)
        v = v[np.abs(v) < 2.0 ** 128]
        np.testing.assert_array_equal(v.astype(np.float32).astype(np.float64), v)

    def bf16_holds(s):
        v = torch.from_numpy(np.ldexp(q, s))
        return torch.equal(v.float().bfloat16().double(), v)

    assert bf16_holds(least) and bf16_holds(0) and not bf16_holds(least - 1)
