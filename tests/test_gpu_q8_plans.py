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
