"""mmbwd_forward_act in bf16 by each of its kernels, the streaming one and the tensor-core
one, whichever of them the sizes would choose: options, activations, values that are not
finite, memory around the outputs, addresses, failed launches, graphs."""
import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm
from test_gpu_epilogue import ACT, check_forward, dev, forward, inputs, lib, no_failed_wait, ok  # noqa: F401 (fixtures)

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("kernel")]
NAN = float("nan")
KERNELS = ["tokens", "tiles"]


@pytest.fixture(params=KERNELS)
def kernel(request, monkeypatch):
    monkeypatch.setenv("MMBWD_ACT_BF16_PATH", request.param)
    return request.param


@pytest.mark.parametrize("T", [1, 31, 64, 129, 300])
@pytest.mark.parametrize("size", [(8, 8), (64, 200), (136, 1000), (1600, 264), (2056, 72)], ids=lambda s: "x".join(map(str, s)))
def test_sizes(T, size):
    x = inputs(T, *size, "bf16")
    first = check_forward(x, "gelu", "bf16")
    for got in (forward(x, "gelu", "bf16"), forward(x, "gelu", "bf16", pre=False, in_place=True)):
        assert torch.equal(got[0], first[0])


@pytest.mark.parametrize("T,C,OC", [(1, 328, 264), (40, 328, 264), (260, 328, 264), (700, 72, 1040)])
@pytest.mark.parametrize("act", ref.ACTS)
def test_activations_and_options(act, T, C, OC):
    for bias in (True, False):
        for residual in (True, False):
            x = inputs(T, C, OC, "bf16", 9, bias, residual)
            full = check_forward(x, act, "bf16")[0]
            assert torch.equal(forward(x, act, "bf16", pre=False)[0], full)
            if residual:
                assert torch.equal(forward(x, act, "bf16", in_place=True)[0], full)
                assert torch.equal(forward(x, act, "bf16", pre=False, in_place=True)[0], full)


@pytest.mark.parametrize("T,C,OC", [(1000, 264, 6416), (2100, 520, 40)])
def test_many_tiles(T, C, OC):
    """More tiles than the streaming kernel has room for at once; several items to a CTA pair."""
    check_forward(inputs(T, C, OC, "bf16", 3), "silu", "bf16")


@pytest.mark.parametrize("T", [7, 200, 300])
def test_non_finite_values_stay_in_their_rows(T):
    x = inputs(T, 264, 136, "bf16", 6)
    clean = forward(x, "gelu", "bf16")[0]
    x["inp"][3, 17], x["inp"][5, 200] = NAN, float("inf")
    bad = forward(x, "gelu", "bf16")[0]
    keep = [i for i in range(T) if i not in (3, 5)]
    assert torch.equal(clean[keep], bad[keep])
    assert torch.isnan(bad[3]).all() and not torch.isfinite(forward(x, "none", "bf16")[0][5]).any()
    x["residual"][6, 2] = NAN
    out = forward(x, "relu", "bf16")[0]
    assert torch.isnan(out[3]).all() and torch.isnan(out[6]).sum() == 1 and not torch.isnan(out[:3]).any()
    x["weight"][9, 4], x["bias"][11] = NAN, float("inf")
    out = forward(x, "none", "bf16")[0]
    assert torch.isnan(out[:, 9]).all() and (out[0, 11] == float("inf")) and not torch.isnan(out[:3, :9]).any()


@pytest.mark.parametrize("act", ref.ACTS)
def test_special_arguments(act):
    """inp . weight^T is 0: the activation of the bias, over every kind of value."""
    vals = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), 1e30, -1e30, NAN, 88.0, -88.0, 10.0, -10.0], dtype=torch.float64)
    bias = ref.rounded(torch.cat([vals, torch.linspace(-25, 25, 333, dtype=torch.float64)]).cuda(), "bf16")
    assert bias.numel() % 8 == 0
    for T in (2, 150):
        x = dict(inp=torch.zeros(T, 64, device="cuda", dtype=torch.float64), weight=torch.ones(bias.numel(), 64, device="cuda", dtype=torch.float64),
                 bias=bias, residual=None)
        out, pre = forward(x, act, "bf16")
        want = ref.act_value(bias, act).expand(T, -1)
        if act in ("gelu", "silu"):
            want = torch.where(bias == -float("inf"), NAN, want)
        bound = ref.stored(ref.act_value_bound(bias, act).expand(T, -1).nan_to_num(0, 0, 0), want, "bf16")
        ref.check(out, want, bound.nan_to_num(0, 0, 0), act)
        assert torch.equal(pre.view(torch.int16)[:, 11:], dev(bias, "bf16").view(torch.int16).expand(T, -1)[:, 11:])


@pytest.mark.parametrize("T", [3, 30, 300])
@pytest.mark.parametrize("C,OC", [(72, 136), (136, 272)])
@pytest.mark.parametrize("shift", [0, 8, 16, 24])
def test_memory_around_the_outputs_and_addresses(T, C, OC, shift):
    """Outputs and residual at every multiple of 16 bytes, in rows that are and are not
    multiples of 32; nothing around them is written."""
    x = inputs(T, C, OC, "bf16", 41)
    want = check_forward(x, "silu", "bf16")
    d = {k: dev(v, "bf16") for k, v in x.items()}
    room = torch.full((3, T * OC + 512), 3.0, device="cuda", dtype=torch.bfloat16)
    lo, hi = 256 + shift, 256 + shift + T * OC
    out, pre, res = (r[lo:hi].view(T, OC) for r in room)
    res.copy_(d["residual"])
    ok(mm.mmbwd_forward_act(out, pre, d["inp"], d["weight"], d["bias"], res, 1, T, C, OC, mm.ACT_SILU, mm.BF16))
    ok(mm.mmbwd_forward_act(res, None, d["inp"], d["weight"], d["bias"], res, 1, T, C, OC, mm.ACT_SILU, mm.BF16))
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1]) and torch.equal(res, want[0])
    assert (room[:, :lo] == 3).all() and (room[:, hi:] == 3).all()


def test_one_tensor_off_a_boundary():
    """One of out, pre and residual between 32-byte boundaries, the others on them."""
    T, C, OC = 300, 136, 272
    x = inputs(T, C, OC, "bf16", 42)
    want = check_forward(x, "gelu", "bf16")
    d = {k: dev(v, "bf16") for k, v in x.items()}
    for off in range(3):
        room = torch.full((3, T * OC + 32), 3.0, device="cuda", dtype=torch.bfloat16)
        out, pre, res = (r[8 if i == off else 0:][:T * OC].view(T, OC) for i, r in enumerate(room))
        res.copy_(d["residual"])
        ok(mm.mmbwd_forward_act(out, pre, d["inp"], d["weight"], d["bias"], res, 1, T, C, OC, mm.ACT_GELU, mm.BF16))
        assert torch.equal(out, want[0]) and torch.equal(pre, want[1]), off


@pytest.mark.parametrize("T", [4, 200])
def test_failed_launches_write_nothing(T):
    d = {k: dev(v, "bf16") for k, v in inputs(T, 64, 64, "bf16").items()}
    out = torch.full((T, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    mm.mmbwd_debug_fail_next_launch(1)
    assert mm.mmbwd_forward_act(out, None, d["inp"], d["weight"], None, None, 1, T, 64, 64, 1, mm.BF16) == mm.ERR_CUDA
    torch.cuda.synchronize()
    assert (out == 9).all()


def test_captured_and_replayed_with_new_inputs():
    T, C, OC = 300, 264, 392
    x, y = inputs(T, C, OC, "bf16", 1), inputs(T, C, OC, "bf16", 50)
    d = {k: dev(v, "bf16") for k, v in x.items()}
    out, pre = torch.empty_like(d["residual"]), torch.empty_like(d["residual"])

    def call():
        ok(mm.mmbwd_forward_act(out, pre, d["inp"], d["weight"], d["bias"], d["residual"], 1, T, C, OC, mm.ACT_GELU, mm.BF16))

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k, v in y.items():
        d[k].copy_(dev(v, "bf16"))
    graph.replay()
    torch.cuda.synchronize()
    want = check_forward(y, "gelu", "bf16")
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1])


@pytest.mark.parametrize("kernel", KERNELS[:1], indirect=True)
def test_the_override_chooses(kernel, monkeypatch):
    """Sums of 6400 products in another order differ somewhere among 100 thousand."""
    x = inputs(64, 6400, 1600, "bf16", 2)
    a = forward(x, "none", "bf16")[0]
    monkeypatch.setenv("MMBWD_ACT_BF16_PATH", "tiles")
    assert not torch.equal(a, forward(x, "none", "bf16")[0])
