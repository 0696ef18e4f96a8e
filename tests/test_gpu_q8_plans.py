"""The 8-bit products' work splits as they are remembered and overridden, on the GPU."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
from test_gpu_q8 import DT, dev, host, lib, normal, q8, tdt  # noqa: F401

pytestmark = pytest.mark.gpu


class Layer:
    """Operands of one backward call, made by the reference."""

    def __init__(self, T, C, OC):
        import torch

        d, inp, w = normal((T, OC), "bf16", 4, 1e-2), normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6, 0.02)
        self.shape = (T, C, OC)
        self.d, self.dt, self.it, self.wt = q8(d, mm.E4M3), q8(d.T, mm.E4M3), q8(inp.T, mm.E4M3), q8(w.T, mm.E4M3)
        self.n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
        self.ws = torch.full((max(self.n, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, dinp, dw, types, add):
        T, C, OC = self.shape
        return mm.mmbwd_q8_backward(dinp, dw, *self.d[:2], *self.dt[:2], *self.it[:2], *self.wt[:2], self.ws, self.n, 1, T,
                                    C, OC, 0, 0, 0, DT[types[0]], DT[types[1]], add)

    def check(self, types=("bf16", "f32"), add=0):
        import torch

        T, C, OC = self.shape
        old = [normal((T, C), types[0], 7), normal((OC, C), types[1], 8)]
        dinp, dw = dev(old[0], types[0]), dev(old[1], types[1])
        assert self.call(dinp, dw, types, add) == mm.OK
        torch.cuda.synchronize()
        want, tol = ref.product_bound(self.d[2], self.wt[2], types[0], old[0] if add & 1 else 0.0)
        assert np.all(np.abs(host(dinp) - want) <= tol)
        want, tol = ref.product_bound(self.dt[2], self.it[2], types[1], old[1] if add & 2 else 0.0)
        assert np.all(np.abs(host(dw) - want) <= tol)


def test_types_and_accumulation_search_no_further_split():
    layer = Layer(900, 264, 392)
    made = mm.mmbwd_q8_debug_plan_searches()
    for types in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")):
        for add in range(4):
            layer.check(types, add)
    assert mm.mmbwd_q8_debug_plan_searches() == made


@pytest.mark.parametrize("shape, splits", [((200, 8200, 26_000), None), ((200, 8200, 26_000), "1,1"),
                                           ((200, 8200, 26_000), "2,1"), ((26_000, 8200, 200), "1,2")],
                         ids=["planned", "unsplit", "dinp split", "dweight split"])
def test_backward_of_more_items_than_the_table_holds(monkeypatch, shape, splits):
    """Over 3000 tiles and splits, which the pairs take in turn: every element is
    written, and sampled elements of every tile, the last ones among them, are right."""
    import torch

    if splits:
        monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    T, C, OC = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(6)

    def operand(R, K, std):
        x = (torch.randn(R, K, generator=g, device="cuda") * std).bfloat16()
        row = (torch.empty(R, ref.ld(K), dtype=torch.uint8, device="cuda"),
               torch.empty(mm.mmbwd_q8_scale_bytes(R, K), dtype=torch.uint8, device="cuda"))
        col = (torch.empty(K, ref.ld(R), dtype=torch.uint8, device="cuda"),
               torch.empty(mm.mmbwd_q8_scale_bytes(K, R), dtype=torch.uint8, device="cuda"))
        assert mm.mmbwd_q8_quantize(*row, *col, None, x, None, 0, R, K, mm.BF16, mm.E4M3) == mm.OK
        return x, row, col

    d, d8, d8t = operand(T, OC, 1e-2)
    x, _, i8t = operand(T, C, 1.0)
    w, _, w8t = operand(OC, C, 0.02)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where a partial sum is missed
    dinp = torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((OC, C), float("nan"), device="cuda")
    assert mm.mmbwd_q8_backward(dinp, dw, *d8, *d8t, *i8t, *w8t, ws, n, 1, T, C, OC, 0, 0, 0, mm.BF16, mm.F32, 0) == mm.OK
    torch.cuda.synchronize()
    assert torch.isfinite(dinp).all() and torch.isfinite(dw).all()

    def some(size, step):  # spread over all 128-wide pieces, and the last two
        return np.r_[np.arange(3, size - 2, step), size - 2, size - 1]

    cols = some(C, 61)
    for got, a, b, rows, dtype in ((dinp, host(d), host(w[:, cols]).T, some(T, 97), "bf16"),
                                   (dw, host(d).T, host(x[:, cols]).T, some(OC, 97), "f32")):
        want, tol = ref.product_bound(ref.quantize(a[rows], mm.E4M3)[2], ref.quantize(b, mm.E4M3)[2], dtype)
        assert np.all(np.abs(host(got[rows][:, cols]) - want) <= tol)


@pytest.mark.parametrize("splits", ["4,1", "1,4"])
def test_one_output_takes_its_own_override(monkeypatch, splits):
    """Each output alone has the bits of a call for both with the same overrides."""
    import torch

    monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    monkeypatch.setenv("MMBWD_Q8_TILE_N", "128,256")
    layer = Layer(1400, 256, 2048)
    (T, C, OC), got = layer.shape, []
    for want in ((1, 1), (1, 0), (0, 1)):
        dinp = torch.full((T, C), float("nan"), device="cuda") if want[0] else None
        dw = torch.full((OC, C), float("nan"), device="cuda") if want[1] else None
        assert layer.call(dinp, dw, ("f32", "f32"), 0) == mm.OK
        got.append((dinp, dw))
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[2][1])
    layer.check()
