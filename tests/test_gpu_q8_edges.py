"""The 8-bit layer and the LayerNorm forward at their edges: nothing written
outside the outputs, operands no call may take, launches that fail, scales whose
product leaves fp32, few tokens in a graph."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
from test_gpu_q8 import DT, dev, host, lib, normal, q8, room, tdt  # noqa: F401

pytestmark = pytest.mark.gpu
BAND = 512  # bytes of sentinel on either side


class Guarded:
    """A buffer of `n` bytes between sentinels."""

    def __init__(self, n, fill=0xC3):
        import torch

        self.n = n
        self.all = torch.full((BAND + -(-n // 256) * 256 + BAND,), 0x5A, dtype=torch.uint8, device="cuda")
        self.at = self.all[BAND:BAND + n]
        self.at.fill_(fill)

    def data_ptr(self):
        return self.at.data_ptr()

    def intact(self):
        import torch

        return bool(torch.all(self.all[:BAND] == 0x5A)) and bool(torch.all(self.all[BAND + self.n:] == 0x5A))

    def as_tensor(self, dtype, *shape):
        return self.at.view(dtype).view(*shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 8), (127, 136), (129, 264), (1030, 1000)], ids=lambda s: "x".join(map(str, s)))
def test_quantize_writes_its_outputs_only(size, dtype):
    import torch

    R, C = size
    es = 2 if dtype == "bf16" else 4
    x = dev(normal((R, C), dtype, 1), dtype)
    n = mm.mmbwd_q8_quantize_workspace_bytes(R, C)
    bufs = [Guarded(k) for k in (mm.mmbwd_q8_data_bytes(R, C), mm.mmbwd_q8_scale_bytes(R, C), mm.mmbwd_q8_data_bytes(C, R),
                                 mm.mmbwd_q8_scale_bytes(C, R), C * es, max(n, 1))]
    assert mm.mmbwd_q8_quantize(*bufs[:5], x, bufs[5], n, R, C, DT[dtype], mm.E4M3) == mm.OK
    torch.cuda.synchronize()
    assert all(b.intact() for b in bufs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(5, 77, 12), (300, 140, 4), (300, 140, 24), (300, 140, 1004), (513, 264, 528), (2500, 136, 640)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forward_bias_at_any_16_bytes(shape, dtype):
    """The bias on 32 bytes and on 16 only, between NaN, with rows of the output on
    32, 16 and 8 bytes: the same results, none of them from outside the bias."""
    import torch

    T, C, OC = shape
    iq, isc, iv = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, wv = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    bias = normal((OC,), dtype, 3)
    want, tol = ref.product_bound(iv, wv, dtype, bias)
    outs = []
    for off in (32, 16):
        room_ = torch.full((OC + 64,), float("nan"), dtype=tdt(dtype), device="cuda")
        first = off // (2 if dtype == "bf16" else 4)
        b = room_[first:first + OC]
        b.copy_(dev(bias, dtype))
        assert b.data_ptr() % 32 == off % 32
        out = torch.full((T, OC), 7.0, dtype=tdt(dtype), device="cuda")
        assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, b, 1, T, C, OC, 0, 0, DT[dtype]) == mm.OK
        torch.cuda.synchronize()
        assert np.all(np.abs(host(out) - want) <= tol)
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", ["128,128", "256,256"])
def test_forward_bias_over_many_tiles(monkeypatch, width, dtype):
    """Several tiles for each CTA pair, the last column of tiles cut: every tile
    adds the bias of its own columns, which is all there is to its result."""
    import torch

    monkeypatch.setenv("MMBWD_Q8_TILE_N", width)
    T, C, OC = 20_100, 8, 1180
    x = torch.zeros(T, C, dtype=tdt(dtype), device="cuda")
    iq, isc, _ = q8(host(x), mm.E4M3)
    wq, wsc, _ = q8(normal((OC, C), dtype, 2), mm.E4M3)
    bias = dev(normal((OC,), dtype, 3), dtype)
    out = torch.full((T + 1, OC), 7.0, dtype=tdt(dtype), device="cuda")
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, bias, 1, T, C, OC, 0, 0, DT[dtype]) == mm.OK
    torch.cuda.synchronize()
    assert torch.equal(out[:T], bias.expand(T, OC))
    assert torch.all(out[T] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 77, 12), (50, 264, 1004), (130, 1160, 136), (300, 140, 1004), (513, 264, 4)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forward_writes_its_output_only(shape, dtype):
    import torch

    T, C, OC = shape
    iq, isc, _ = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, _ = q8(normal((OC, C), "bf16", 2), mm.E4M3)
    out = Guarded(T * OC * (2 if dtype == "bf16" else 4), fill=0xFF)
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, T, C, OC, 0, 0, DT[dtype]) == mm.OK
    torch.cuda.synchronize()
    assert out.intact()
    assert torch.all(torch.isfinite(out.as_tensor(tdt(dtype), T, OC)))


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("splits", ["0,0", "2,3"])
@pytest.mark.parametrize("shape", [(1, 4, 12), (300, 260, 131), (700, 1032, 264)], ids=lambda s: "x".join(map(str, s)))
def test_backward_writes_its_outputs_only(monkeypatch, shape, types, splits):
    import torch

    monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    T, C, OC = shape
    d, inp, w = normal((T, OC), "bf16", 4), normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6)
    dq, ds, _ = q8(d, mm.E4M3)
    dqt, dst, _ = q8(d.T, mm.E4M3)
    iqt, ist, _ = q8(inp.T, mm.E4M3)
    wqt, wst, _ = q8(w.T, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    es = {"bf16": 2, "f32": 4}
    ws, dinp, dw = Guarded(max(n, 1)), Guarded(T * C * es[types[0]], 0xFF), Guarded(OC * C * es[types[1]], 0xFF)
    assert mm.mmbwd_q8_backward(dinp, dw, dq, ds, dqt, dst, iqt, ist, wqt, wst, ws, n, 1, T, C, OC, 0, 0, 0,
                                DT[types[0]], DT[types[1]], 0) == mm.OK
    torch.cuda.synchronize()
    assert ws.intact() and dinp.intact() and dw.intact()
    assert torch.all(torch.isfinite(dinp.as_tensor(tdt(types[0]), T, C)))
    assert torch.all(torch.isfinite(dw.as_tensor(tdt(types[1]), OC, C)))


@pytest.mark.parametrize("size", [(1, 8), (5, 264), (9, 2400), (7, 8200), (3, 65544)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_forward_writes_its_outputs_only(size):
    import torch

    T, C = size
    x, w = dev(normal((T, C), "bf16", 1), "bf16"), dev(normal((C,), "bf16", 2), "bf16")
    out, mean, rstd = Guarded(T * C * 2), Guarded(T * 4), Guarded(T * 4)
    assert mm.lnbwd_forward(out, mean, rstd, x, w, None, 1, T, C, 1e-5, mm.BF16) == mm.OK
    torch.cuda.synchronize()
    assert out.intact() and mean.intact() and rstd.intact()


def test_refused_and_failed_calls_leave_everything_as_it_was():
    import torch

    T, C, OC = 40, 264, 136
    x = dev(normal((T, C), "bf16", 1), "bf16")
    q, s = room(T, C)
    qt, st = room(C, T)
    wq, wsc, _ = q8(normal((OC, C), "bf16", 2), mm.E4M3)
    out = torch.full((T, OC), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((C, C), 7.0, device="cuda")
    host_x = torch.zeros(T, C, dtype=torch.bfloat16)
    assert mm.mmbwd_q8_quantize(q, s, qt, st, None, host_x, None, 0, T, C, mm.BF16, 0) == mm.ERR_MEMORY
    pinned = torch.zeros(T, C, dtype=torch.bfloat16).pin_memory()
    assert mm.mmbwd_q8_quantize(q, s, qt, st, None, pinned, None, 0, T, C, mm.BF16, 0) == mm.ERR_MEMORY
    calls = [lambda: mm.mmbwd_q8_quantize(q, s, qt, st, None, x, None, 0, T, C, mm.BF16, 0),
             lambda: mm.mmbwd_q8_forward(out, q, s, wq, wsc, None, 1, T, C, OC, 0, 0, mm.BF16),
             lambda: mm.mmbwd_q8_backward(None, dw, None, None, qt, st, qt, st, None, None, None, 0, 1, T, C, C, 0, 0, 0,
                                          mm.BF16, mm.F32, 0),
             lambda: mm.lnbwd_forward(out, None, None, out, wq, None, 1, T, OC, 1e-5, mm.BF16)]
    for call in calls:
        mm.mmbwd_debug_fail_next_launch(1)
        assert call() == mm.ERR_CUDA
    mm.mmbwd_debug_fail_next_launch(0)
    torch.cuda.synchronize()
    assert torch.all(q == 0xA5) and torch.all(s == 0xFF) and torch.all(qt == 0xA5) and torch.all(st == 0xFF)
    assert torch.all(out == 7.0) and torch.all(dw == 7.0)
    assert [c() for c in calls[:3]] == [mm.OK] * 3  # and the next call works
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [3, 300])
def test_scales_whose_product_leaves_fp32(tokens):
    """Blocks scaled so far up (or down) that the product of two scales is beyond
    fp32: where no nonzero values meet, the sum is zero, not a NaN; where they
    meet far below fp32, zero; beyond its top, an infinity."""
    import torch

    C, OC = 256, 8
    x, w = np.zeros((tokens, C)), np.zeros((OC, C))
    x[0, 0], x[0, 128] = 2.0 ** 126, 1.0
    x[1, 0], x[1, 130] = 2.0 ** -100, 2.0
    x[2, 0], x[2, 131] = 2.0 ** 100, 3.0
    w[0, 5], w[0, 128], w[0, 130], w[0, 131] = 2.0 ** 120, 1.0, 1.0, 1.0  # meets x in the second block only
    w[1, 0], w[1, 128], w[1, 130], w[1, 131] = 2.0 ** -100, 1.0, 1.0, 1.0
    w[2, 0] = 2.0 ** 60
    iq, isc, iv = q8(x, mm.E4M3)
    wq, wsc, wv = q8(w, mm.E4M3)
    assert np.array_equal(iv, x) and np.array_equal(wv, w)
    out = torch.empty(tokens, OC, device="cuda")
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, tokens, C, OC, 0, 0, mm.F32) == mm.OK
    torch.cuda.synchronize()
    got = host(out)
    assert got[0, 0] == 1.0 and got[1, 0] == 2.0 and got[2, 0] == 3.0
    # (2^26 + 1 needs 27 bits: in fp32 it is 2^26; 2^-200 + 2 is 2)
    assert got[0, 1] == 2.0 ** 26 and got[1, 1] == 2.0 and got[2, 1] == 4.0
    assert got[0, 2] == np.inf and got[1, 2] == 2.0 ** -40 and got[2, 2] == np.inf
    assert np.all(got[3:] == 0.0) and np.all(got[:, 3:] == 0.0)


def test_few_tokens_in_a_graph():
    import torch

    T, C, OC = 5, 1600, 520
    w8 = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    x = dev(normal((T, C), "bf16", 1), "bf16")
    q, s = room(T, C)
    out = torch.empty(T, OC, dtype=torch.bfloat16, device="cuda")

    def call(o):
        assert mm.mmbwd_q8_quantize(q, s, None, None, None, x, None, 0, T, C, mm.BF16, 0) == mm.OK
        assert mm.mmbwd_q8_forward(o, q, s, w8[0], w8[1], None, 1, T, C, OC, 0, 0, mm.BF16) == mm.OK

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    call(out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(3):
            call(out)
    y = normal((T, C), "bf16", 9)
    x.copy_(dev(y, "bf16"))
    out.fill_(float("nan"))
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    want, tol = ref.product_bound(ref.quantize(y, mm.E4M3)[2], w8[2], "bf16")
    assert np.all(np.abs(host(out) - want) <= tol)


def test_gradients_against_differences():
    """L = sum of dout * out is linear in each coordinate of inp and weight, so
    L(x + e_k) - L(x) is the gradient exactly. Whole numbers up to 8 are exact in
    either format and direction, and every sum is exact in fp32."""
    import torch

    T, C, OC = 70, 136, 72
    g = np.random.default_rng(5)
    inp, w, d = (g.integers(-4, 5, s).astype(float) for s in ((T, C), (OC, C), (T, OC)))

    def forms(x):
        R, K = x.shape
        a, b = room(R, K), room(K, R)
        assert mm.mmbwd_q8_quantize(*a, *b, None, dev(x, "f32"), None, 0, R, K, mm.F32, mm.E4M3) == mm.OK
        return a, b

    def loss(x, v):
        out = torch.empty(T, OC, device="cuda")
        assert mm.mmbwd_q8_forward(out, *forms(x)[0], *forms(v)[0], None, 1, T, C, OC, 0, 0, mm.F32) == mm.OK
        return float((host(out) * d).sum())

    dinp, dw, db = torch.empty(T, C, device="cuda"), torch.empty(OC, C, device="cuda"), torch.empty(OC, device="cuda")
    a, b = room(T, OC), room(OC, T)
    assert mm.mmbwd_q8_quantize(*a, *b, db, dev(d, "f32"), None, 0, T, OC, mm.F32, mm.E4M3) == mm.OK
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    assert mm.mmbwd_q8_backward(dinp, dw, *a, *b, *forms(inp)[1], *forms(w)[1], ws, n, 1, T, C, OC, 0, 0, 0, mm.F32,
                                mm.F32, 0) == mm.OK
    torch.cuda.synchronize()
    at = loss(inp, w)
    for r, c in ((0, 0), (69, 135), (3, 127), (40, 128), (17, 64)):
        x = inp.copy()
        x[r, c] += 1
        assert loss(x, w) - at == host(dinp)[r, c]
    for r, c in ((0, 0), (71, 135), (5, 127), (64, 128), (31, 9)):
        v = w.copy()
        v[r, c] += 1
        assert loss(inp, v) - at == host(dw)[r, c]
    np.testing.assert_array_equal(host(db), d.sum(0))  # L is affine in a bias with slope sum of dout


def test_calls_from_several_threads_at_once():
    """Threads with a stream and buffers each, calling at the same time: every
    result is the one a single call gives."""
    import threading

    import torch

    from test_gpu_q8 import _Buffers, _layer

    T, C, OC = 600, 520, 392
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    made = []
    for _ in range(3):
        x = [torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, C), (OC, C), (T, OC))]
        made.append((x, _Buffers(T, C, OC), torch.cuda.Stream(), [t.clone() for t in _layer(*x)]))
    torch.cuda.synchronize()
    wrong = []

    def work(x, b, stream, want):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = _layer(*x, b)
                stream.synchronize()
                wrong.extend(i for i, (p, q) in enumerate(zip(got, want)) if not torch.equal(p, q))

    threads = [threading.Thread(target=work, args=m) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
