"""The global gradient norm and clipping on the GPU against 64 bits."""
import math

import pytest
import torch

import block_reference as ref
import linear_layer_gemms_gb300 as mm

pytestmark = pytest.mark.gpu
DT = {"bf16": mm.BF16, "f32": mm.F32}
NAN = float("nan")
# A thread sums 64 squares in fp32 (each off by two roundings, the sums by up to 20 more in
# four chains), all else is 64 bits; the root halves that and rounds once: 12 steps of 2^-24.
NORM_REL = 12 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mm.load()


def ok(rc):
    assert rc == mm.OK, mm.strerror(rc)


def room(rows):
    return torch.full((mm.mmbwd_grad_workspace_bytes(len(rows)),), 0xFF, device="cuda", dtype=torch.uint8)


def entry(g, out=None):
    return g, out, g.numel(), mm.BF16 if g.dtype == torch.bfloat16 else mm.F32


def exact_norm(ts):
    # scaled, so that no square leaves the range of 64 bits
    top = max([t.double().abs().max().item() for t in ts if t.numel()] + [0.0])
    if not top or math.isinf(top) or math.isnan(top):
        return top
    return top * math.sqrt(sum((t.double() / top).square().sum().item() for t in ts))


def norm_of(ts):
    rows = [entry(t) for t in ts]
    out = torch.full((1,), NAN, device="cuda")
    ws = room(rows)
    ok(mm.mmbwd_grad_norm(out, mm.grad_list(rows), ws, ws.numel()))
    return out


def clip(ts, outs, max_norm):
    rows = [entry(t, o) for t, o in zip(ts, outs)]
    norm = torch.full((1,), NAN, device="cuda")
    ws = room(rows)
    ok(mm.mmbwd_grad_clip(norm, mm.grad_list(rows), max_norm, ws, ws.numel()))
    return norm


def check_norm(got, ts):
    want = exact_norm(ts)
    assert abs(got.item() - want) <= NORM_REL * want, (got.item(), want)


def coefficient(norm, max_norm):
    """What the definition gives in fp32 from the norm that was stored."""
    f = torch.tensor([max_norm], dtype=torch.float32) / (norm.cpu() + torch.tensor(1e-6))
    return torch.where(f < 1, f, torch.where(torch.isnan(f), f, torch.ones(1))).item()


def scaled(t, coef):
    return (t.float() * torch.tensor(coef, device="cuda", dtype=torch.float32)).to(t.dtype)


def same(a, b):
    v = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    nan = torch.isnan(a) & torch.isnan(b)
    return bool(((a.view(v) == b.view(v)) | nan).all())


def some(n, dtype, seed, std=0.01, offset=0):
    """n values that start `offset` elements after a 16-byte boundary, between guards."""
    flat = torch.full((n + offset + 64,), 3.0, device="cuda", dtype=ref.TDT[dtype])
    flat[offset:offset + n] = ref.normal(seed, n, std=std).to(ref.TDT[dtype])
    return flat[offset:offset + n]


SIZES = [1, 2, 3, 5, 7, 8, 9, 15, 17, 255, 2047, 4097, 8191, 8192, 8193, 16383, 16384, 16385, 16393, 100003]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", SIZES)
def test_one_tensor(n, dtype):
    """Sizes around a vector, a block's chunk and several, at every alignment of both sides."""
    for a in range(0, 8 if dtype == "bf16" else 4):
        t = some(n, dtype, n + a, offset=a)
        norm = norm_of([t])
        check_norm(norm, [t])
        for b in (a, (a + 3) % (8 if dtype == "bf16" else 4)):
            out = some(n, dtype, 1, offset=b)
            limit = norm.item() * 0.3
            got = clip([t], [out], limit)
            assert torch.equal(got, norm)
            assert same(out, scaled(t, coefficient(norm, limit)))
            base = out._base if out._base is not None else out
            assert (base[:b] == 3).all() and (base[b + n:] == 3).all()
        want = scaled(t, coefficient(norm, limit))
        clip([t], [None], limit)
        assert same(t, want)
        base = t._base
        assert (base[:a] == 3).all() and (base[a + n:] == 3).all()


def test_many_tensors_of_both_types():
    """More than one launch holds, empty ones among them, in place and out of place mixed."""
    ts, outs = [], []
    for i in range(2500):
        n = [0, 1, 3, 17, 64, 257, 1000, 33000][i % 8] + (i % 5 if i % 8 else 0)
        ts.append(some(n, "bf16" if i % 3 else "f32", i, offset=i % 4))
        outs.append(torch.full_like(ts[-1], NAN) if i % 2 else None)
    norm = norm_of(ts)
    check_norm(norm, ts)
    before = [t.clone() for t in ts]
    limit = norm.item() / 7
    assert torch.equal(clip(ts, outs, limit), norm)
    coef = coefficient(norm, limit)
    for t, o, b in zip(ts, outs, before):
        assert same(t if o is None else o, scaled(b, coef))
        assert o is None or same(t, b)


def test_under_the_limit():
    """In place nothing is written; other buffers get the values as they are."""
    ts = [some(1000, "bf16", 1), some(777, "f32", 2, offset=1)]
    outs = [None, torch.full_like(ts[1], NAN)]
    before = [t.clone() for t in ts]
    norm = exact_norm(ts)
    for limit in (norm * 1.01, 3e38):
        clip(ts, outs, limit)
        assert same(ts[0], before[0]) and same(outs[1], before[1])
    got = clip(ts, outs, norm * 0.999)
    coef = coefficient(got, norm * 0.999)
    # (bf16 neighbours are 2^-8 to 2^-7 apart, relatively: 0.999 is less than half a step off and changes none)
    assert coef < 1 and same(ts[0], scaled(before[0], coef)) and same(ts[0], before[0])
    assert same(outs[1], scaled(ts[1], coef)) and not same(outs[1], ts[1])


def test_no_limit_at_all_and_zero():
    ts = [some(100, "f32", 1)]
    clip(ts, [None], 0.0)
    assert not ts[0].any()
    z = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.bfloat16)]
    assert norm_of(z).item() == 0.0
    clip(z, [None, None], 1.0)
    assert not z[0].any() and not z[1].any()
    assert norm_of([]).item() == 0.0
    empty = torch.empty(0, device="cuda")
    assert norm_of([empty, empty]).item() == 0.0
    got = clip([empty], [None], 1.0)
    assert got.item() == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-22, 1e-13, 1e-9, 1e10, 1e18, 1e20, 1e30, 1e36])
def test_values_whose_squares_leave_fp32(std, dtype):
    ts = [some(5000, dtype, 5, std=std), some(9, dtype, 6, std=std, offset=1)]
    check_norm(norm_of(ts), ts)
    mixed = ts + [some(3000, "f32", 7, std=1.0)]
    check_norm(norm_of(mixed), mixed)
    # one large value among ordinary ones, and one ordinary value among zeros
    t = some(20000, dtype, 8)
    t[12345] = 1e25
    check_norm(norm_of([t]), [t])
    t.zero_()
    t[777] = 1e-30
    check_norm(norm_of([t]), [t])


def test_infinities_and_nans():
    ts = [some(500, "f32", 1), some(400, "bf16", 2)]
    ts[1][7] = -float("inf")
    outs = [torch.empty_like(t) for t in ts]
    norm = clip(ts, outs, 1.0)
    assert norm.item() == float("inf")
    assert not outs[0].any() and torch.isnan(outs[1][7]) and not outs[1][8:].any()
    ts[0][3] = NAN
    norm = clip(ts, outs, 1.0)
    assert math.isnan(norm.item()) and torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()
    big = [torch.full((64,), 3e38, device="cuda")]  # a norm beyond fp32
    assert norm_of(big).item() == float("inf")


def test_a_given_norm():
    """The norm of two lists joined by the program, then each list scaled."""
    a, b = [some(3000, "bf16", 1), some(70, "f32", 2)], [some(999, "f32", 3)]
    joined = (norm_of(a).double().square() + norm_of(b).double().square()).sqrt().float()
    limit = joined.item() * 0.5
    want = [scaled(t, coefficient(joined, limit)) for t in a + b]
    for ts in (a, b):
        ok(mm.mmbwd_grad_scale(mm.grad_list([entry(t) for t in ts]), joined, limit))
    for t, w in zip(a + b, want):
        assert same(t, w)


def test_a_tensor_twice_counts_twice():
    t = some(5000, "bf16", 4)
    assert abs(norm_of([t, t]).item() - math.sqrt(2) * exact_norm([t])) <= NORM_REL * 2 * exact_norm([t])


def test_large_tensors_and_repeats():
    """More chunks than blocks, the same bits on every call."""
    ts = [torch.empty(30_000_001, device="cuda", dtype=torch.bfloat16).normal_(0, 0.01), torch.empty(20_000_003, device="cuda").normal_(0, 0.01)]
    first = norm_of(ts)
    want = math.sqrt(sum(t.double().square().sum().item() for t in ts))
    assert abs(first.item() - want) <= NORM_REL * want
    for _ in range(5):
        assert torch.equal(norm_of(ts), first)
    limit = want * 0.25
    outs = [torch.empty_like(t) for t in ts]
    clip(ts, outs, limit)
    coef = coefficient(first, limit)
    for t, o in zip(ts, outs):
        assert same(o, scaled(t, coef))
    clip(ts, [None, None], limit)
    for t, o in zip(ts, outs):
        assert same(o, t)


def test_captured_and_on_two_streams():
    lists = [[some(40000, "bf16", 10 * i), some(5001, "f32", 10 * i + 1)] for i in range(2)]
    outs = [[torch.empty_like(t) for t in ts] for ts in lists]
    limit = 0.5 * exact_norm(lists[0])
    want = []
    for ts in lists:
        o = [torch.empty_like(t) for t in ts]
        want.append((clip(ts, o, limit), o))
    rows = [mm.grad_list([entry(t, o) for t, o in zip(ts, os)]) for ts, os in zip(lists, outs)]
    ws = [room(r) for r in rows]
    norms = [torch.empty(1, device="cuda") for _ in rows]
    streams = [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            ok(mm.mmbwd_grad_clip(norms[i], rows[i], limit, ws[i], ws[i].numel(), stream=s.cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(norms[i], want[i][0]) and all(same(a, b) for a, b in zip(outs[i], want[i][1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        ok(mm.mmbwd_grad_clip(norms[0], rows[0], limit, ws[0], ws[0].numel()))
    del rows  # the list's entries travelled with the launches
    for t, n in zip(lists[0], lists[1]):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norms[0], want[1][0]) and all(same(a, b) for a, b in zip(outs[0], want[1][1]))


def test_failed_launches_and_host_memory():
    t = some(1000, "f32", 1)
    norm = torch.full((1,), 9.0, device="cuda")
    ws = room([0])
    mm.mmbwd_debug_fail_next_launch(1)
    assert mm.mmbwd_grad_clip(norm, mm.grad_list([entry(t)]), 1e-6, ws, ws.numel()) == mm.ERR_CUDA
    torch.cuda.synchronize()
    assert norm.item() == 9.0
    assert mm.mmbwd_grad_norm(norm, mm.grad_list([entry(torch.zeros(5))]), ws, ws.numel()) == mm.ERR_MEMORY
    assert mm.mmbwd_grad_norm(torch.zeros(1), mm.grad_list([entry(t)]), ws, ws.numel()) == mm.ERR_MEMORY


def test_a_tensor_of_more_than_2_31_values():
    n = 2 ** 31 + 12345
    t = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    t[0], t[2 ** 31 + 3], t[n - 1] = 2.0, 1.0, 2.0
    norm = torch.full((1,), float("nan"), device="cuda")
    ws_bytes = mm.mmbwd_grad_workspace_bytes(1)
    ws = torch.empty(ws_bytes, device="cuda", dtype=torch.uint8)
    lst = mm.grad_list([(t, None, n, mm.BF16)])
    assert mm.mmbwd_grad_clip(norm, lst, 1.5, ws, ws_bytes) == mm.OK
    assert norm.item() == 3.0  # sums of squares that are exact
    # (1.5 / 3.000001 rounds to 0.5 in bf16's eight bits)
    assert t[0] == 1.0 and t[2 ** 31 + 3] == 0.5 and t[n - 1] == 1.0 and torch.count_nonzero(t) == 3
