"""The 8-bit linear layer on the GPU against numpy in 64 bits: quantisation bit
for bit, products within the bound of their sums (tests/q8_reference.py)."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import q8_reference as ref
import synth

pytestmark = pytest.mark.gpu
DT = {"bf16": mm.BF16, "f32": mm.F32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()
    yield
    assert mm.mmbwd_device_status()[0] == mm.OK


def tdt(dtype):
    import torch

    return torch.bfloat16 if dtype == "bf16" else torch.float32


def dev(a: np.ndarray, dtype: str):
    """float64 values that the type holds exactly, on the device in that type."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(tdt(dtype)).cuda()


def host(t) -> np.ndarray:
    return t.double().cpu().numpy()


def normal(shape, dtype, seed, std=1.0):
    """Seeded values, rounded to `dtype`, as float64."""
    a = synth.normal(shape, dtype, seed, 1, 0.0, std)
    return synth.to_f64(a, dtype)


def room(rows, K):
    """Buffers of an 8-bit matrix, filled with bytes that must all be overwritten."""
    import torch

    return (torch.full((rows, ref.ld(K)), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((mm.mmbwd_q8_scale_bytes(rows, K),), 0xFF, dtype=torch.uint8, device="cuda"))


def quantize(x: np.ndarray, dtype, fmt, row=True, col=True, sums=False):
    import torch

    R, C = x.shape
    q, s = room(R, C) if row else (None, None)
    qt, st = room(C, R) if col else (None, None)
    cs = torch.full((C,), 3.0, dtype=tdt(dtype), device="cuda") if sums else None
    n = mm.mmbwd_q8_quantize_workspace_bytes(R, C) if sums else 0
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda") if sums else None
    rc = mm.mmbwd_q8_quantize(q, s, qt, st, cs, dev(x, dtype), ws, n, R, C, DT[dtype], fmt)
    assert rc == mm.OK, mm.strerror(rc)
    torch.cuda.synchronize()
    return q, s, qt, st, cs


def same_bits(q, s, x, fmt):
    want_q, want_s, value = ref.quantize(x, fmt)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    return value


def q8(x, fmt):
    """Operand in 8-bit form made by the reference: device buffers and values."""
    import torch

    bits, scales, value = ref.quantize(x, fmt)
    return torch.from_numpy(bits).cuda(), torch.from_numpy(scales).cuda(), value


SIZES = [(1, 8), (1, 1600), (7, 128), (33, 136), (127, 120), (128, 512), (129, 264), (300, 1000), (777, 520), (1024, 136),
         (1025, 264), (2500, 72)]


@pytest.mark.parametrize("fmt", [mm.E4M3, mm.E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_quantize_is_exact(size, dtype, fmt):
    R, C = size
    x = normal((R, C), dtype, seed=R * 1000 + C) * np.exp2(np.arange(C) % 7 - 3.0)
    x[::5] = 0.0  # rows without a nonzero value
    x[:, 3::11] = 0.0
    q, s, qt, st, cs = quantize(x, dtype, fmt, sums=True)
    same_bits(q, s, x, fmt)
    same_bits(qt, st, x.T, fmt)
    # fp32 sums: at most 8 + 1 + 8 + ceil(blocks / 8) + 8 additions deep
    depth = 25 + -(-(-(-R // 128)) // 8)
    tol = depth * 2.0 ** -24 * np.abs(x).sum(0)
    want = x.sum(0)
    assert np.all(np.abs(host(cs) - want) <= tol + ref.HALF_STEP[dtype] * (np.abs(want) + tol))


@pytest.mark.parametrize("forms", [(True, False), (False, True)], ids=["row", "column"])
def test_quantize_one_form(forms):
    x = normal((200, 392), "bf16", seed=5)
    q, s, qt, st, _ = quantize(x, "bf16", mm.E4M3, row=forms[0], col=forms[1], sums=forms[1])
    if forms[0]:
        same_bits(q, s, x, mm.E4M3)
    else:
        same_bits(qt, st, x.T, mm.E4M3)


@pytest.mark.parametrize("fmt", [mm.E4M3, mm.E5M2], ids=["e4m3", "e5m2"])
def test_quantize_borders(fmt):
    """Block maxima on both sides of the format's largest value at every
    exponent, halfway values, values that leave a subnormal, the ends of fp32."""
    emax, mant, emin, _ = ref.FORMAT[fmt]
    top = 1.75 * 2.0 ** emax
    rows = []
    for p in range(-149, 128, 3):
        for f in (1.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), np.float32(2) - np.float32(2.0 ** -23)):
            m = np.float32(np.ldexp(float(f), p))
            if np.isfinite(m) and m > 0:
                r = np.zeros(128)
                r[5] = -float(m)
                r[6:70] = float(m) * np.linspace(0, 1, 64)
                rows.append(r)
    for k in range(64):  # halfway between neighbours, with the block's maximum at the top
        r = np.zeros(128)
        r[0] = top
        r[1:65] = np.ldexp((np.arange(64) + 0.5), emin - mant + k % 12)
        rows.append(np.minimum(r, top))
    rows.append(np.full(128, float(np.finfo(np.float32).max)))
    x = np.array(rows).astype(np.float32).astype(np.float64)
    q, s, qt, st, _ = quantize(x, "f32", fmt)
    same_bits(q, s, x, fmt)
    same_bits(qt, st, x.T, fmt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_non_finite_values_become_nan_alone(dtype):
    x = normal((140, 264), dtype, seed=9)
    x[3, 7], x[3, 9], x[60, 200], x[139, 263] = np.inf, np.nan, -np.inf, np.nan
    x[100] = np.nan  # a row, and a column, of nothing finite
    x[:, 50] = np.inf
    q, s, qt, st, _ = quantize(x, dtype, mm.E4M3)
    same_bits(q, s, x, mm.E4M3)
    same_bits(qt, st, x.T, mm.E4M3)


def test_quantize_empty():
    import torch

    cs = torch.full((64,), 5.0, device="cuda")
    assert mm.mmbwd_q8_quantize(None, None, None, None, cs, None, None, 0, 0, 64, mm.F32, mm.E4M3) == mm.OK
    torch.cuda.synchronize()
    assert torch.all(cs == 0)
    assert mm.mmbwd_q8_quantize(None, None, None, None, None, None, None, 0, 5, 0, mm.F32, mm.E4M3) == mm.OK


def test_quantize_offsets_beyond_32_bits():
    """A matrix whose bytes pass 2^32 in x and in both forms: its last tiles."""
    import torch

    R, C = 4_200_007, 1032
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    tail = normal((300, C), "bf16", seed=4)
    x[-300:] = dev(tail, "bf16")
    q = torch.empty(R, ref.ld(C), dtype=torch.uint8, device="cuda")
    s = torch.empty(mm.mmbwd_q8_scale_bytes(R, C), dtype=torch.uint8, device="cuda")
    qt = torch.empty(C, ref.ld(R), dtype=torch.uint8, device="cuda")
    st = torch.empty(mm.mmbwd_q8_scale_bytes(C, R), dtype=torch.uint8, device="cuda")
    assert q.numel() > 1 << 32 and qt.numel() > 1 << 32
    assert mm.mmbwd_q8_quantize(q, s, qt, st, None, x, None, 0, R, C, mm.BF16, mm.E4M3) == mm.OK
    torch.cuda.synchronize()
    want, _, _ = ref.quantize(tail, mm.E4M3)
    np.testing.assert_array_equal(q[-300:].cpu().numpy(), want)
    first = (R - 300) // 128 * 128  # whole blocks of rows, zeros before the tail
    block = np.zeros((R - first, C))
    block[-300:] = tail
    want_t, _, _ = ref.quantize(block.T, mm.E4M3)
    np.testing.assert_array_equal(qt[:, first:].cpu().numpy(), want_t)
    del x, q, qt
    torch.cuda.empty_cache()


# (tokens, C, OC): single tokens, short and odd prompts, ragged in every direction
SHAPES = [(1, 8, 8), (1, 1600, 520), (2, 264, 136), (5, 24, 1000), (16, 768, 2304), (17, 1000, 264), (48, 640, 328),
          (64, 136, 4104), (100, 520, 392), (129, 128, 128), (130, 1160, 136), (255, 392, 776), (300, 2056, 264),
          (777, 264, 1032), (100, 264, 10_008), (200, 392, 5000), (257, 1032, 24), (300, 140, 1004),
          (3, 77, 12), (400, 1001, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    import torch

    T, C, OC = shape
    fi, fw = (mm.E4M3, mm.E5M2) if T % 2 else (mm.E4M3, mm.E4M3)
    iq, isc, iv = q8(normal((T, C), dtype, 1), fi)
    wq, wsc, wv = q8(normal((OC, C), dtype, 2, 0.02), fw)
    for bias in (None, normal((OC,), dtype, 3)):
        out = torch.full((T + 1, OC), 7.0, dtype=tdt(dtype), device="cuda")  # one row behind the last
        b = None if bias is None else dev(bias, dtype)
        rc = mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, b, 1, T, C, OC, fi, fw, DT[dtype])
        assert rc == mm.OK, mm.strerror(rc)
        torch.cuda.synchronize()
        want, tol = ref.product_bound(iv, wv, dtype, 0.0 if bias is None else bias)
        assert np.all(np.abs(host(out[:T]) - want) <= tol)
        assert torch.all(out[T] == 7.0)


@pytest.mark.parametrize("splits", ["1", "2", "4", "8"])
@pytest.mark.parametrize("shape", [(1, 1032, 264), (7, 2056, 520), (16, 1160, 132), (31, 1800, 260), (33, 1096, 392),
                                   (64, 1032, 1000), (65, 1032, 264), (130, 1160, 392), (256, 1096, 136)], ids=lambda s: "x".join(map(str, s)))
def test_forward_few_tokens_every_split(monkeypatch, shape, splits):
    """Few tokens: K shared by 1 to 8 CTAs, partial tiles of tokens and rows."""
    import torch

    monkeypatch.setenv("MMBWD_Q8_TOKEN_SPLITS", splits)
    T, C, OC = shape
    iq, isc, iv = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, wv = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    for dtype in ("f32", "bf16"):
        bias = normal((OC,), dtype, 3)
        out = torch.full((T + 1, OC), 7.0, dtype=tdt(dtype), device="cuda")
        for _ in range(2):
            assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, dev(bias, dtype), 1, T, C, OC, 0, 0, DT[dtype]) == mm.OK
        torch.cuda.synchronize()
        want, tol = ref.product_bound(iv, wv, dtype, bias)
        assert np.all(np.abs(host(out[:T]) - want) <= tol)
        assert torch.all(out[T] == 7.0)


@pytest.mark.parametrize("T", [1, 20, 50])
def test_forward_few_tokens_many_tiles(T):
    """More tiles than CTAs: each CTA walks several."""
    import torch

    C, OC = 264, 80_040
    iq, isc, iv = q8(normal((T, C), "bf16", 1), mm.E4M3)
    wq, wsc, wv = q8(normal((OC, C), "bf16", 2, 0.02), mm.E4M3)
    out = torch.empty(T, OC, dtype=torch.bfloat16, device="cuda")
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, T, C, OC, 0, 0, mm.BF16) == mm.OK
    torch.cuda.synchronize()
    want, tol = ref.product_bound(iv, wv, "bf16")
    assert np.all(np.abs(host(out) - want) <= tol)


BACKWARD = [(1, 8, 8), (3, 264, 136), (128, 128, 128), (200, 328, 520), (500, 136, 264), (300, 1032, 24),
  (1000, 264, 392),
            (130, 520, 2304), (300, 260, 131), (77, 1044, 25), (600, 4, 1001)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("shape", BACKWARD, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, types):
    import torch

    T, C, OC = shape
    fd = mm.E5M2 if T % 3 == 0 else mm.E4M3
    d = normal((T, OC), "bf16", 4, 1e-2)
    d[::7] = 0.0  # tokens that carry no gradient
    inp, w = normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6, 0.02)
    dq, ds, dv = q8(d, fd)
    dqt, dst, dvt = q8(d.T, fd)
    iqt, ist, ivt = q8(inp.T, mm.E4M3)
    wqt, wst, wvt = q8(w.T, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    old = [normal((T, C), types[0], 7), normal((OC, C), types[1], 8)]
    for add in (0, mm.Q8_ADD_DINP, mm.Q8_ADD_DWEIGHT, 3):
        dinp, dw = dev(old[0], types[0]), dev(old[1], types[1])
        rc = mm.mmbwd_q8_backward(dinp, dw, dq, ds, dqt, dst, iqt, ist, wqt, wst, ws, n, 1, T, C, OC, fd, mm.E4M3,
                                  mm.E4M3, DT[types[0]], DT[types[1]], add)
        assert rc == mm.OK, mm.strerror(rc)
        torch.cuda.synchronize()
        want, tol = ref.product_bound(dv, wvt, types[0], old[0] if add & 1 else 0.0)
        assert np.all(np.abs(host(dinp) - want) <= tol)
        want, tol = ref.product_bound(dvt, ivt, types[1], old[1] if add & 2 else 0.0)
        assert np.all(np.abs(host(dw) - want) <= tol)


@pytest.mark.parametrize("tiles", ["256,256", "128,128", "128,256"])
@pytest.mark.parametrize("splits", ["1,1", "2,3", "4,1", "1,8"])
def test_backward_splits_and_tile_widths(monkeypatch, splits, tiles):
    """Every tile width and split count the planner may take gives the result,
    in one order of additions."""
    import torch

    monkeypatch.setenv("MMBWD_Q8_SPLITS", splits)
    monkeypatch.setenv("MMBWD_Q8_TILE_N", tiles)
    T, C, OC = 1400, 392, 1096
    d, inp, w = normal((T, OC), "bf16", 4, 1e-2), normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6, 0.02)
    dq, ds, dv = q8(d, mm.E4M3)
    dqt, dst, dvt = q8(d.T, mm.E4M3)
    iqt, ist, ivt = q8(inp.T, mm.E4M3)
    wqt, wst, wvt = q8(w.T, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    assert (n > 0) == (splits != "1,1")
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    old = [normal((T, C), "bf16", 7), normal((OC, C), "f32", 8)]
    for add in (0, 3):
        got = []
        for _ in range(2):
            dinp, dw = dev(old[0], "bf16"), dev(old[1], "f32")
            assert mm.mmbwd_q8_backward(dinp, dw, dq, ds, dqt, dst, iqt, ist, wqt, wst, ws, n, 1, T, C, OC, 0, 0, 0,
                                        mm.BF16, mm.F32, add) == mm.OK
            torch.cuda.synchronize()
            got.append((dinp, dw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        want, tol = ref.product_bound(dv, wvt, "bf16", old[0] if add else 0.0)
        assert np.all(np.abs(host(got[0][0]) - want) <= tol)
        want, tol = ref.product_bound(dvt, ivt, "f32", old[1] if add else 0.0)
        assert np.all(np.abs(host(got[0][1]) - want) <= tol)


def test_backward_one_output_only():
    import torch

    T, C, OC = 200, 264, 392
    d, inp, w = normal((T, OC), "bf16", 4, 1e-2), normal((T, C), "bf16", 5), normal((OC, C), "bf16", 6, 0.02)
    dq, ds, dv = q8(d, mm.E4M3)
    dqt, dst, dvt = q8(d.T, mm.E4M3)
    iqt, ist, ivt = q8(inp.T, mm.E4M3)
    wqt, wst, wvt = q8(w.T, mm.E4M3)
    n = mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    dinp, dw = (torch.full((r, C), 9.0, dtype=torch.bfloat16, device="cuda") for r in (T, OC))
    tail = (ws, n, 1, T, C, OC, mm.E4M3, mm.E4M3, mm.E4M3, mm.BF16, mm.BF16, 0)
    assert mm.mmbwd_q8_backward(dinp, None, dq, ds, None, None, None, None, wqt, wst, *tail) == mm.OK
    assert mm.mmbwd_q8_backward(None, dw, None, None, dqt, dst, iqt, ist, None, None, *tail) == mm.OK
    torch.cuda.synchronize()
    for got, (want, tol) in ((dinp, ref.product_bound(dv, wvt, "bf16")), (dw, ref.product_bound(dvt, ivt, "bf16"))):
        assert np.all(np.abs(host(got) - want) <= tol)


def test_empty_sums():
    import torch

    out = torch.full((3, 16), 4.0, device="cuda")
    b = dev(normal((16,), "f32", 3), "f32")
    assert mm.mmbwd_q8_forward(out, None, None, None, None, b, 1, 3, 0, 16, 0, 0, mm.F32) == mm.OK
    torch.cuda.synchronize()
    assert torch.equal(out, b.expand(3, 16))
    dw = torch.full((16, 8), 4.0, device="cuda")
    args = (None, None, None, None, None, None, None, None, None, 0, 1, 0, 8, 16, 0, 0, 0, mm.F32, mm.F32)
    assert mm.mmbwd_q8_backward(None, dw, *args, mm.Q8_ADD_DWEIGHT) == mm.OK
    torch.cuda.synchronize()
    assert torch.all(dw == 4.0)
    assert mm.mmbwd_q8_backward(None, dw, *args, 0) == mm.OK
    torch.cuda.synchronize()
    assert torch.all(dw == 0.0)


def test_extreme_scales_and_nan_stay_in_their_rows():
    """Rows of the largest and the smallest magnitudes beside ordinary ones, and
    a NaN, which reaches the results of its own row and no other."""
    import torch

    T, C, OC = 140, 264, 136
    x, w = normal((T, C), "f32", 1), normal((OC, C), "f32", 2)
    x[10] *= 2.0 ** 100
    x[11] *= 2.0 ** -110
    w[5] *= 2.0 ** -100
    w[6] *= 2.0 ** 20
    x[70, 200] = np.nan
    iq, isc, iv = q8(x, mm.E4M3)
    wq, wsc, wv = q8(w, mm.E4M3)
    out = torch.empty(T, OC, device="cuda")
    assert mm.mmbwd_q8_forward(out, iq, isc, wq, wsc, None, 1, T, C, OC, 0, 0, mm.F32) == mm.OK
    torch.cuda.synchronize()
    got = host(out)
    assert np.all(np.isnan(got[70]))
    keep = np.arange(T) != 70
    want, tol = ref.product_bound(iv[keep], wv, "f32")
    # a product of scales under 2^-126 may leave fp32's normal range
    assert np.all(np.abs(got[keep] - want) <= tol + 2.0 ** -126 * C)


@pytest.mark.parametrize("shape", [(1, 1600, 4800), (16, 768, 1024), (777, 768, 2304), (2048, 1600, 1600)],
                         ids=lambda s: "x".join(map(str, s)))
def test_repeated_calls_give_the_same_bits(shape):
    import torch

    T, C, OC = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    w = torch.randn(OC, C, generator=g, device="cuda").bfloat16()
    d = (torch.randn(T, OC, generator=g, device="cuda") * 0.01).bfloat16()
    got = []
    for _ in range(3):
        got.append(_layer(x, w, d))
        torch.cuda.synchronize()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def _forms(x):
    import torch

    R, C = x.shape
    q, s = torch.empty(R, ref.ld(C), dtype=torch.uint8, device="cuda"), torch.empty(mm.mmbwd_q8_scale_bytes(R, C), dtype=torch.uint8, device="cuda")
    qt, st = torch.empty(C, ref.ld(R), dtype=torch.uint8, device="cuda"), torch.empty(mm.mmbwd_q8_scale_bytes(C, R), dtype=torch.uint8, device="cuda")
    return q, s, qt, st


class _Buffers:
    def __init__(self, T, C, OC):
        import torch

        self.x8, self.w8, self.d8 = (_forms(torch.empty(s, device="meta")) for s in ((T, C), (OC, C), (T, OC)))
        n = max(mm.mmbwd_q8_quantize_workspace_bytes(T, OC), mm.mmbwd_q8_backward_workspace_bytes(1, T, C, OC))
        self.n, self.ws = n, torch.empty(n, dtype=torch.uint8, device="cuda")
        self.out = torch.empty(T, OC, dtype=torch.bfloat16, device="cuda")
        self.dinp = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
        self.dw = torch.empty(OC, C, device="cuda")
        self.db = torch.empty(OC, dtype=torch.bfloat16, device="cuda")


def _layer(x, w, d, b=None):
    """The 8-bit layer's forward and backward on the current stream."""
    (T, C), OC = x.shape, w.shape[0]
    b = b or _Buffers(T, C, OC)
    ok = []
    ok.append(mm.mmbwd_q8_quantize(*b.x8, None, x, None, 0, T, C, mm.BF16, mm.E4M3))
    ok.append(mm.mmbwd_q8_quantize(*b.w8, None, w, None, 0, OC, C, mm.BF16, mm.E4M3))
    ok.append(mm.mmbwd_q8_forward(b.out, *b.x8[:2], *b.w8[:2], None, 1, T, C, OC, 0, 0, mm.BF16))
    ok.append(mm.mmbwd_q8_quantize(*b.d8, b.db, d, b.ws, b.n, T, OC, mm.BF16, mm.E5M2))
    ok.append(mm.mmbwd_q8_backward(b.dinp, b.dw, *b.d8, *b.x8[2:], *b.w8[2:], b.ws, b.n, 1, T, C, OC, mm.E5M2, mm.E4M3,
                                   mm.E4M3, mm.BF16, mm.F32, 0))
    assert ok == [mm.OK] * 5, ok
    return b.out, b.dinp, b.dw, b.db


def test_graphs_streams_and_their_own_workspaces():
    """Two captured graphs of the layer replayed at the same time on two
    streams, with new inputs in place, give the eager calls' bits."""
    import torch

    T, C, OC = 1000, 392, 520
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def inputs():
        return ((torch.randn(T, C, generator=g, device="cuda")).bfloat16(),
                (torch.randn(OC, C, generator=g, device="cuda") * 0.02).bfloat16(),
                (torch.randn(T, OC, generator=g, device="cuda") * 0.01).bfloat16())

    made = []
    for _ in range(2):
        x, b = inputs(), _Buffers(T, C, OC)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            _layer(*x, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            _layer(*x, b)
        made.append((x, b, s, graph))
    for x, _, _, _ in made:
        for t, new in zip(x, inputs()):
            t.copy_(new)
    want = [[t.clone() for t in _layer(*x)] for x, _, _, _ in made]
    for _, b, _, _ in made:
        for t in (b.out, b.dinp, b.dw, b.db):
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for _, _, s, graph in made:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, b, _, _), w in zip(made, want):
        for got, t in zip((b.out, b.dinp, b.dw, b.db), w):
            assert torch.equal(got, t)


def test_forward_offsets_beyond_32_bits():
    """An output of more than 2^32 elements: rows at its end."""
    import torch

    T, C, OC = 131_080, 64, 33_000
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    w = torch.randn(OC, C, generator=g, device="cuda").bfloat16()
    x8, w8 = _forms(x), _forms(w)
    assert mm.mmbwd_q8_quantize(*x8, None, x, None, 0, T, C, mm.BF16, mm.E4M3) == mm.OK
    assert mm.mmbwd_q8_quantize(*w8, None, w, None, 0, OC, C, mm.BF16, mm.E4M3) == mm.OK
    out = torch.zeros(T, OC, dtype=torch.bfloat16, device="cuda")
    assert out.numel() > 1 << 32
    assert mm.mmbwd_q8_forward(out, *x8[:2], *w8[:2], None, 1, T, C, OC, 0, 0, mm.BF16) == mm.OK
    torch.cuda.synchronize()
    iv = ref.quantize(host(x[-50:]), mm.E4M3)[2]
    wv = ref.quantize(host(w), mm.E4M3)[2]
    want, tol = ref.product_bound(iv, wv, "bf16")
    assert np.all(np.abs(host(out[-50:]) - want) <= tol)
    del out
    torch.cuda.empty_cache()


def test_layer_norm_into_the_8_bit_layer_and_back():
    """The operators as a GPT-2 block uses them: LayerNorm forward, its output
    quantised (checkpoint kept), the 8-bit product; then dout quantised with
    dbias, the 8-bit backward, and the LayerNorm backward from the forward's
    statistics. Every stage against 64 bits of its own inputs."""
    import torch

    T, C, OC = 260, 392, 520
    x, gamma, beta = normal((T, C), "bf16", 1), 1 + 0.25 * normal((C,), "bf16", 2), normal((C,), "bf16", 3)
    gamma = host(dev(gamma, "bf16"))
    w, bias, d = normal((OC, C), "bf16", 4, 0.02), normal((OC,), "bf16", 5), normal((T, OC), "bf16", 6, 1e-2)
    ln = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    gx, gg, gb = dev(x, "bf16"), dev(gamma, "bf16"), dev(beta, "bf16")
    assert mm.lnbwd_forward(ln, mean, rstd, gx, gg, gb, 1, T, C, 1e-5, mm.BF16) == mm.OK
    b = _Buffers(T, C, OC)
    gw, gd, gbias = dev(w, "bf16"), dev(d, "bf16"), dev(bias, "bf16")
    assert mm.mmbwd_q8_quantize(*b.x8, None, ln, None, 0, T, C, mm.BF16, mm.E4M3) == mm.OK
    assert mm.mmbwd_q8_quantize(*b.w8, None, gw, None, 0, OC, C, mm.BF16, mm.E4M3) == mm.OK
    assert mm.mmbwd_q8_forward(b.out, *b.x8[:2], *b.w8[:2], gbias, 1, T, C, OC, 0, 0, mm.BF16) == mm.OK
    assert mm.mmbwd_q8_quantize(*b.d8, b.db, gd, b.ws, b.n, T, OC, mm.BF16, mm.E4M3) == mm.OK
    assert mm.mmbwd_q8_backward(b.dinp, b.dw, *b.d8, *b.x8[2:], *b.w8[2:], b.ws, b.n, 1, T, C, OC, 0, 0, 0, mm.BF16,
                                mm.F32, 0) == mm.OK
    dx = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    dgamma, dbeta = torch.zeros(C, dtype=torch.bfloat16, device="cuda"), torch.zeros(C, dtype=torch.bfloat16, device="cuda")
    assert mm.lnbwd_run(dx, dgamma, dbeta, b.dinp, gx, gg, mean, rstd, 1, T, C, mm.BF16) == mm.OK
    torch.cuda.synchronize()

    m, v = x.mean(1), x.var(1)
    r = 1 / np.sqrt(v + 1e-5)
    want = (x - m[:, None]) * r[:, None] * gamma + beta
    assert np.all(np.abs(host(ln) - want) <= ref.HALF_STEP["bf16"] * np.abs(want) + 1e-5 * (np.abs(want) + np.abs(beta) + 1))
    a = host(ln)
    iv, ivt = ref.quantize(a, mm.E4M3)[2], ref.quantize(a.T, mm.E4M3)[2]
    wv, wvt = ref.quantize(w, mm.E4M3)[2], ref.quantize(w.T, mm.E4M3)[2]
    dv, dvt = ref.quantize(d, mm.E4M3)[2], ref.quantize(d.T, mm.E4M3)[2]
    for got, (ex, tol) in ((b.out, ref.product_bound(iv, wv, "bf16", bias)), (b.dinp, ref.product_bound(dv, wvt, "bf16")),
                           (b.dw, ref.product_bound(dvt, ivt, "f32"))):
        assert np.all(np.abs(host(got) - ex) <= tol)
    dy = host(b.dinp)
    n = (x - m[:, None]) * r[:, None]
    gy = dy * gamma
    ex = r[:, None] * (gy - gy.mean(1, keepdims=True) - n * (gy * n).mean(1, keepdims=True))
    rms = np.sqrt(np.mean(ex ** 2))
    assert np.all(np.abs(host(dx) - ex) <= 2e-2 * (np.abs(ex) + rms))
