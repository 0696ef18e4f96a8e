"""The 8-bit products at a training step's sizes against 64 bits: several items of
many blocks to each CTA pair, so that both overlapping accumulators are used again
and again. Every column of sampled rows, the rows from both halves and all
lane quadrants of every row tile."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
from test_gpu_q8 import DT, dev, host, lib, tdt  # noqa: F401

pytestmark = pytest.mark.gpu


def operand(R, K, std, seed, fmt):
    """Seeded bf16 values and their row and column forms, by the library (which are
    bit for bit the reference's: tests/test_gpu_q8.py)."""
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(R, K, generator=g, device="cuda") * std).bfloat16()
    row = (torch.empty(R, ref.ld(K), dtype=torch.uint8, device="cuda"),
           torch.empty(mm.mmbwd_q8_scale_bytes(R, K), dtype=torch.uint8, device="cuda"))
    col = (torch.empty(K, ref.ld(R), dtype=torch.uint8, device="cuda"),
           torch.empty(mm.mmbwd_q8_scale_bytes(K, R), dtype=torch.uint8, device="cuda"))
    assert mm.mmbwd_q8_quantize(*row, *col, None, x, None, 0, R, K, mm.BF16, fmt) == mm.OK
    return x, row, col


def rows_of(size):  # 37 is odd: all quadrants in turn, three or four rows of each 128
    return np.r_[np.arange(5, size, 37), size - 1]


def check(got, a, b, dtype, extra=0.0):
    want, tol = ref.product_bound(a, b, dtype, extra)
    bad = np.abs(host(got) - want) > tol
    assert not bad.any(), f"{bad.sum()} elements, first at {np.argwhere(bad)[0]}"


# (tokens, C, OC): GPT-2 XL's fc (10 items a pair), a short reduction (two blocks) and a
# ragged one with as many
SHAPES = [(8192, 1600, 6400), (8192, 256, 6400), (5000, 520, 9976)]


@pytest.mark.parametrize("width", [None, "128,128", "256,256"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(monkeypatch, shape, width):
    import torch

    if width:
        monkeypatch.setenv("MMBWD_Q8_TILE_N", width)
    T, C, OC = shape
    x, x8, _ = operand(T, C, 1.0, 1, mm.E4M3)
    w, w8, _ = operand(OC, C, 0.02, 2, mm.E4M3)
    bias = torch.linspace(-1, 1, OC, device="cuda")
    rows = rows_of(T)
    iv, wv = ref.quantize(host(x[rows]), mm.E4M3)[2], ref.quantize(host(w), mm.E4M3)[2]
    for dtype in ("f32", "bf16"):
        b = bias.to(tdt(dtype))
        out = torch.full((T, OC), float("nan"), dtype=tdt(dtype), device="cuda")
        assert mm.mmbwd_q8_forward(out, *x8, *w8, b, 1, T, C, OC, 0, 0, DT[dtype]) == mm.OK
        torch.cuda.synchronize()
        assert torch.isfinite(out).all()
        check(out[rows], iv, wv, dtype, host(b))


@pytest.mark.parametrize("width", [None, "128,256", "256,128"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(monkeypatch, shape, width):
    """Both products in one launch, of one width and of two; dweight overwritten and
    added to."""
    import torch

    if width:
        monkeypatch.setenv("MMBWD_Q8_TILE_N", width)
    T, C, OC = shape
    d, d8, d8t = operand(T, OC, 1e-2, 3, mm.E5M2)
    x, _, x8t = operand(T, C, 1.0, 4, mm.E4M3)
    w, _, w8t = operand(OC, C, 0.02, 5, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    rt, ro = rows_of(T), rows_of(OC)
    dv, wv = ref.quantize(host(d[rt]), mm.E5M2)[2], ref.quantize(host(w).T, mm.E4M3)[2]
    dvt, xv = ref.quantize(host(d[:, ro]).T, mm.E5M2)[2], ref.quantize(host(x).T, mm.E4M3)[2]
    old = torch.linspace(-3, 3, OC * C, device="cuda").view(OC, C)
    for wtype, add in (("f32", mm.Q8_ADD_DWEIGHT), ("bf16", 0)):
        dinp = torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
        dw = old.clone() if add else torch.full((OC, C), float("nan"), dtype=tdt(wtype), device="cuda")
        assert mm.mmbwd_q8_backward(dinp, dw, *d8, *d8t, *x8t, *w8t, ws, n, 1, T, C, OC, mm.E5M2, 0, 0, mm.BF16, DT[wtype],
                                    add) == mm.OK
        torch.cuda.synchronize()
        assert torch.isfinite(dinp).all() and torch.isfinite(dw).all()
        check(dinp[rt], dv, wv, "bf16")
        check(dw[ro], dvt, xv, wtype, host(old[ro]) if add else 0.0)
