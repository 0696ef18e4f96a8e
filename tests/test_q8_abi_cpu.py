"""Refusals and sizes of the 8-bit linear layer and the LayerNorm forward,
without a GPU; and the reference that the GPU tests use, against torch."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_layer_gemms_gb300 import _build

    _build.build()
    mm.load()


A = 1 << 24  # fake, aligned addresses: validation fails before any use


def test_sizes():
    assert mm.mmbwd_q8_data_bytes(3, 100) == 3 * 112
    assert mm.mmbwd_q8_scale_bytes(1, 1) == 512 and mm.mmbwd_q8_scale_bytes(129, 513) == 2 * 2 * 512
    assert mm.mmbwd_q8_data_bytes(0, 100) == 0 and mm.mmbwd_q8_scale_bytes(5, 0) == 0
    assert mm.mmbwd_q8_data_bytes(-1, 100) == 0 and mm.mmbwd_q8_scale_bytes(5, 1 << 31) == 0
    assert mm.mmbwd_q8_data_bytes(1 << 22, 2048) == 1 << 33
    assert mm.mmbwd_q8_quantize_workspace_bytes(1025, 64) == 9 * 64 * 4 and mm.mmbwd_q8_quantize_workspace_bytes(1024, 64) == 0
    assert mm.mmbwd_q8_quantize_workspace_bytes(-1, 64) == 0
    assert mm.mmbwd_q8_backward_workspace_bytes(-1, 8, 64, 64) == 0


def quantize(**kw):
    a = dict(q=A, scale=2 * A, qt=3 * A, scale_t=4 * A, colsum=5 * A, x=6 * A, workspace=7 * A, workspace_bytes=1 << 20,
             rows=100, cols=64, dtype=mm.BF16, format=mm.E4M3, stream=0)
    a.update(kw)
    return mm.mmbwd_q8_quantize(**a)


def test_quantize_refusals():
    assert quantize(dtype=2) == mm.ERR_DTYPE
    assert quantize(format=2) == mm.ERR_DTYPE
    assert quantize(rows=-1) == mm.ERR_SHAPE
    assert quantize(cols=1 << 31) == mm.ERR_SHAPE
    assert quantize(rows=1 << 30, cols=1 << 30) == mm.ERR_SHAPE
    assert quantize(x=None) == mm.ERR_NULL
    assert quantize(scale=None) == mm.ERR_NULL
    assert quantize(qt=None) == mm.ERR_NULL
    assert quantize(q=None, scale=None, qt=None, scale_t=None) == mm.ERR_NULL
    assert quantize(workspace=None, rows=2000) == mm.ERR_NULL
    assert quantize(workspace_bytes=8, rows=2000) == mm.ERR_SHAPE
    assert quantize(workspace=7 * A + 16, rows=2000) == mm.ERR_ALIGN
    assert quantize(x=6 * A + 8) == mm.ERR_ALIGN
    assert quantize(cols=60) == mm.ERR_ALIGN
    assert quantize(q=6 * A + 64) == mm.ERR_ALIAS
    assert quantize(scale=A + 6400 - 16) == mm.ERR_ALIAS
    assert quantize(colsum=7 * A, rows=2000) == mm.ERR_ALIAS
    assert quantize(colsum=6 * A) == mm.ERR_ALIAS


def forward(**kw):
    a = dict(out=A, inp_q=2 * A, inp_scale=3 * A, weight_q=4 * A, weight_scale=5 * A, bias=6 * A, B=2, T=8, C=60, OC=32,
             inp_format=mm.E4M3, weight_format=mm.E4M3, dtype=mm.BF16, stream=0)
    a.update(kw)
    return mm.mmbwd_q8_forward(**a)


def test_forward_refusals():
    assert forward(dtype=5) == mm.ERR_DTYPE
    assert forward(inp_format=-1) == mm.ERR_DTYPE
    assert forward(weight_format=2) == mm.ERR_DTYPE
    assert forward(T=-1) == mm.ERR_SHAPE
    assert forward(B=1 << 20, T=1 << 20) == mm.ERR_SHAPE
    assert forward(out=None) == mm.ERR_NULL
    assert forward(weight_scale=None) == mm.ERR_NULL
    assert forward(OC=34) == mm.ERR_ALIGN
    assert forward(inp_scale=3 * A + 4) == mm.ERR_ALIGN
    assert forward(out=4 * A + 16) == mm.ERR_ALIAS
    assert forward(bias=A + 32) == mm.ERR_ALIAS


def backward(**kw):
    a = dict(dinp=A, dweight=2 * A, dout_q=3 * A, dout_scale=4 * A, dout_qt=5 * A, dout_scale_t=6 * A, inp_qt=7 * A,
             inp_scale_t=8 * A, weight_qt=9 * A, weight_scale_t=10 * A, workspace=11 * A, workspace_bytes=1 << 23, B=2, T=8,
             C=64, OC=40, dout_format=mm.E5M2, inp_format=mm.E4M3, weight_format=mm.E4M3, dinp_dtype=mm.BF16,
             dweight_dtype=mm.F32, accumulate=0, stream=0)
    a.update(kw)
    return mm.mmbwd_q8_backward(**a)


def test_backward_refusals():
    assert backward(dinp_dtype=3) == mm.ERR_DTYPE
    assert backward(dweight_dtype=3) == mm.ERR_DTYPE
    assert backward(dout_format=9) == mm.ERR_DTYPE
    assert backward(accumulate=4) == mm.ERR_SHAPE
    assert backward(OC=-8) == mm.ERR_SHAPE
    assert backward(dinp=None, dweight=None) == mm.ERR_NULL
    assert backward(weight_qt=None) == mm.ERR_NULL
    assert backward(inp_scale_t=None) == mm.ERR_NULL
    assert backward(C=62) == mm.ERR_ALIGN
    assert backward(dinp=A + 8) == mm.ERR_ALIGN
    assert backward(dweight=A + 64) == mm.ERR_ALIAS
    assert backward(dinp=9 * A) == mm.ERR_ALIAS
    need = mm.mmbwd_q8_backward_workspace_bytes(2, 8, 64, 40)
    if need:
        assert backward(workspace_bytes=need - 1) == mm.ERR_SHAPE
        assert backward(workspace=None) == mm.ERR_NULL


def test_an_impossible_override_falls_back_to_the_planner(monkeypatch):
    """A forced split that needs more items than the schedule holds is dropped:
    the plan is the unforced one, never one left over from another shape."""
    shape = (8, 1024, 1600, 6400)
    want = mm.mmbwd_q8_backward_workspace_bytes(*shape)
    for T in range(1, 40):  # plans of other shapes, with workspaces of their own
        monkeypatch.setenv("MMBWD_Q8_SPLITS", "1,2")
        assert mm.mmbwd_q8_backward_workspace_bytes(T, 1024, 264, 392) > 0
    monkeypatch.setenv("MMBWD_Q8_SPLITS", "16,16")
    monkeypatch.setenv("MMBWD_Q8_TILE_N", "128,128")
    assert mm.mmbwd_q8_backward_workspace_bytes(*shape) == want


def layernorm(**kw):
    a = dict(out=A, mean=2 * A, rstd=3 * A, inp=4 * A, weight=5 * A, bias=6 * A, B=2, T=8, C=64, eps=1e-5, dtype=mm.BF16,
             stream=0)
    a.update(kw)
    return mm.lnbwd_forward(**a)


def test_layernorm_forward_refusals():
    assert layernorm(dtype=2) == mm.ERR_DTYPE
    assert layernorm(C=(1 << 20) + 8) == mm.ERR_SHAPE
    assert layernorm(eps=-1.0) == mm.ERR_SHAPE
    assert layernorm(eps=float("nan")) == mm.ERR_SHAPE
    assert layernorm(eps=float("inf")) == mm.ERR_SHAPE
    assert layernorm(weight=None) == mm.ERR_NULL
    assert layernorm(inp=None) == mm.ERR_NULL
    assert layernorm(C=60) == mm.ERR_ALIGN
    assert layernorm(mean=2 * A + 2) == mm.ERR_ALIGN
    assert layernorm(inp=A + 64) == mm.ERR_ALIAS
    assert layernorm(rstd=2 * A + 32) == mm.ERR_ALIAS
    assert layernorm(mean=A + 128) == mm.ERR_ALIAS


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_a_gpu_fail_cleanly():
    for call in (quantize, forward, backward, layernorm):
        assert call() in (mm.ERR_CUDA, mm.ERR_ARCH)
    assert layernorm(out=4 * A) in (mm.ERR_CUDA, mm.ERR_ARCH)  # in place is allowed


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.E5M2])
def test_reference_formats_against_torch(fmt):
    import torch

    f8 = torch.float8_e4m3fn if fmt == ref.E4M3 else torch.float8_e5m2
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(f8).double().numpy()
    np.testing.assert_array_equal(ref.decode(bits, fmt), want)
    top = 448.0 if fmt == ref.E4M3 else 57344.0
    y = np.concatenate([np.linspace(-top, top, 4001), np.ldexp(np.linspace(-1, 1, 999), -12)]).astype(np.float32)
    np.testing.assert_array_equal(ref.encode(y.astype(float), fmt), torch.from_numpy(y).to(f8).view(torch.uint8).numpy())


def test_reference_quantize_by_hand():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 129] = 448.0, -1.0, 3.0
    x[1, 5] = 449.0
    bits, scales, value = ref.quantize(x, ref.E4M3)
    assert bits.shape == (2, 144) and scales.size == 512
    # row 0: 448 fits with s = 0; 3 in the second block is 3 * 2^7 = 384 with s = -7
    assert scales[0] == 127 and scales[1] == 127 - 7 and scales[16] == 128 and scales[17] == 127
    assert value[0, 0] == 448 and value[0, 1] == -1 and value[0, 129] == 3 and value[1, 5] == 448
    assert not bits[:, 130:].any()
