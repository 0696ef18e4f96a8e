"""The LayerNorm forward on the GPU against numpy in 64 bits."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
import synth

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": mm.BF16, "f32": mm.F32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()


def dev(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def host(t):
    return t.double().cpu().numpy()


def normal(shape, dtype, seed, std=1.0):
    return synth.to_f64(synth.normal(shape, dtype, seed, 1, 0.0, std), dtype)


def expected(x, w, b, eps, dtype):
    """(mean, rstd, out) and how far each may be. The mean of C fp32 values: a
    sum at most C / 32 + 16 additions deep, each off by 2^-24 of the magnitudes'
    sum, and three more roundings. The variance's relative error is twice that of
    a difference (x - mean) plus as many roundings, rstd's half of it plus four;
    out multiplies (x - mean) by rstd and the weight and adds the bias."""
    C = x.shape[1]
    deep = C / 32 + 16
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    u = 2.0 ** -24
    e_mean = (deep + 3) * u * np.abs(x).mean(1)
    # each (x - mean) is off by e_mean + u |x - mean|: on the variance
    e_var = (deep + 6) * u * var + e_mean ** 2 + 2 * e_mean * np.abs(x - mean[:, None]).mean(1)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * u)
    n = (x - mean[:, None]) * rstd[:, None]
    out = n * w + b
    e_out = np.abs(w) * (e_mean[:, None] * rstd[:, None] + np.abs(x - mean[:, None]) * e_rstd[:, None]
                         + 4 * u * np.abs(n)) + 2 * u * (np.abs(n * w) + np.abs(b))
    return (mean, e_mean), (rstd, e_rstd), (out, e_out + HALF_STEP[dtype] * (np.abs(out) + e_out))


def call(x, w, b, eps, dtype, stats=True, in_place=False):
    import torch

    T, C = x.shape
    gx = dev(x, dtype)
    out = gx if in_place else torch.full_like(gx, float("nan"))
    mean = torch.full((T,), float("nan"), device="cuda") if stats else None
    rstd = torch.full((T,), float("nan"), device="cuda") if stats else None
    rc = mm.lnbwd_forward(out, mean, rstd, gx, dev(w, dtype), None if b is None else dev(b, dtype), 1, T, C, eps, DT[dtype])
    assert rc == mm.OK, mm.strerror(rc)
    torch.cuda.synchronize()
    return out, mean, rstd


# widths of every kernel variant, their borders, and ragged ones
WIDTHS = [8, 64, 264, 768, 1024, 1032, 1600, 2048, 2056, 4096, 4104, 6400, 8192, 8200, 16384, 16392, 32768, 32776,
          65544]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS)
def test_against_64_bits(C, dtype):
    T = 37 if C <= 8192 else 5
    x = normal((T, C), dtype, C) + np.linspace(-3, 3, T)[:, None]
    x = host(dev(x, dtype))
    x[1] = 2.5  # a row without variance
    x[2] = 0.0
    w, b = normal((C,), dtype, C + 1), normal((C,), dtype, C + 2)
    out, mean, rstd = call(x, w, b, 1e-5, dtype)
    for got, (want, tol) in zip((mean, rstd, out), expected(x, w, b, 1e-5, dtype)):
        assert np.all(np.abs(host(got) - want) <= tol)


@pytest.mark.parametrize("size", [(1, 520), (2, 520), (7, 520), (4099, 520), (4099, 2400), (2500, 6400)],
                         ids=lambda s: "x".join(map(str, s)))
def test_rows(size):
    """One row, less than a block of rows, and many to each team."""
    T, C = size
    x, w, b = normal((T, C), "bf16", T), normal((C,), "bf16", 1), normal((C,), "bf16", 2)
    out, mean, rstd = call(x, w, b, 1e-5, "bf16")
    for got, (want, tol) in zip((mean, rstd, out), expected(x, w, b, 1e-5, "bf16")):
        assert np.all(np.abs(host(got) - want) <= tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [264, 1600, 65544])
def test_without_bias_or_statistics_and_in_place(C, dtype):
    x, w = normal((9, C), dtype, 3), normal((C,), dtype, 4)
    want, tol = expected(x, w, 0.0, 1e-5, dtype)[2]
    got = [host(call(x, w, None, 1e-5, dtype, stats=s, in_place=p)[0]) for s, p in ((True, False), (False, False), (True, True))]
    for g in got:
        assert np.all(np.abs(g - want) <= tol)
        np.testing.assert_array_equal(g, got[0])


def test_a_large_mean_costs_no_precision():
    """Rows far from zero: the variance comes from the differences."""
    x = normal((16, 768), "f32", 5) + 4096.0
    x = host(dev(x, "f32"))
    w, b = np.ones(768), np.zeros(768)
    out, mean, rstd = call(x, w, b, 1e-5, "f32")
    for got, (want, tol) in zip((mean, rstd, out), expected(x, w, b, 1e-5, "f32")):
        assert np.all(np.abs(host(got) - want) <= tol)


def test_non_finite_values_stay_in_their_rows():
    x, w, b = normal((12, 264), "bf16", 6), normal((264,), "bf16", 7), normal((264,), "bf16", 8)
    y = x.copy()
    y[3, 17], y[8, 200] = np.nan, np.inf
    clean, bad = call(x, w, b, 1e-5, "bf16")[0], call(y, w, b, 1e-5, "bf16")[0]
    keep = [i for i in range(12) if i not in (3, 8)]
    np.testing.assert_array_equal(host(bad)[keep], host(clean)[keep])
    assert np.all(np.isnan(host(bad)[[3, 8]]))


def test_captured_and_replayed_with_new_inputs():
    import torch

    T, C = 64, 768
    x, w, b = (dev(normal(s, "bf16", k), "bf16") for k, s in enumerate(((T, C), (C,), (C,))))
    out, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        assert mm.lnbwd_forward(out, mean, rstd, x, w, b, 1, T, C, 1e-5, mm.BF16) == mm.OK
    x.copy_(dev(normal((T, C), "bf16", 99), "bf16"))
    want = torch.empty_like(x)
    assert mm.lnbwd_forward(want, None, None, x, w, b, 1, T, C, 1e-5, mm.BF16) == mm.OK
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
