"""Norms, clipping and scaling of lists of tensors against plain sums in fp64.

Bounds.  Eight squares are summed in fp32: a square, a fused multiply-add and two additions, four
roundings of relative 2^-24 on a sum of non-negative terms; the root halves that, the result is
rounded once more: a norm is off by at most 3 x 2^-24.  The factor adds a sum and a quotient: 5 x 2^-24.
A scaled element is the correctly rounded product of its value and the factor: equal bits.
"""
import math

import pytest
import torch

import newton_schulz_hyperball_b200 as nshb

pytestmark = pytest.mark.gpu
DEV = "cuda"
NORM_TOL, FACTOR_TOL = 3 * 2.0 ** -24, 5 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make(shapes, dtype, seed=0, scale=1.0):
    g = gen(seed)
    return [(torch.randn(s, generator=g, device=DEV) * scale).to(dtype) for s in shapes]


def exact_norms(ts, kind=nshb.NSHB_NORM_L2):
    if kind == nshb.NSHB_NORM_INF:
        each = [float(t.double().abs().max()) if t.numel() else 0.0 for t in ts]
        return max(each, default=0.0), each
    sq = [float(t.double().square().sum()) for t in ts]
    return math.sqrt(math.fsum(sq)), [math.sqrt(s) for s in sq]


def norm(ts, max_norm=1.0, kind=nshb.NSHB_NORM_L2, want_each=True, handle=None):
    h = handle or nshb.tensors(ts)
    ws = nshb.tensor_workspace(h).fill_(0xAB)
    total = torch.full((2,), -1.0, device=DEV)
    each = torch.full((max(len(ts), 1),), -1.0, device=DEV) if want_each else None
    nshb.grad_norm(h, total, ws, max_norm=max_norm, each=each, kind=kind)
    return total, each, nshb.device_status(ws)


def close(got, want, tol):
    return abs(got - want) <= tol * abs(want)


SETS = {
    "one element": [(1,)],
    "one short vector": [(7,)],
    "one window": [(4096,)],
    "one window and one": [(8193,)],
    "a window for each group": [(4096,)] * 32,
    "one more": [(4096,)] * 33,
    "short ones and empty ones": [(0,), (100,), (0, 3), (9000,), (50, 60)],
    "vectors": [(128,), (2048,), (1,), (33,), (4097,)] * 5,
    "matrices": [(64, 64), (5, 7), (768, 768), (1, 9), (300, 700), (130, 1)],
    "a large one": [(2048, 2049), (3,)],
    "with empty ones": [(0,), (5, 3), (0, 4), (17,), (4, 0)],
    "more than a launch": [(1 + i % 50,) for i in range(1100)],
    "empty ones fill a launch": [(0,)] * 600 + [(10,)] * 3,
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("kind", [nshb.NSHB_NORM_L2, nshb.NSHB_NORM_INF])
def test_norms(name, dtype, kind):
    ts = make(SETS[name], dtype, seed=len(name))
    want, want_each = exact_norms(ts, kind)
    total, each, flags = norm(ts, max_norm=0.5, kind=kind)
    alone, _, _ = norm(ts, max_norm=0.5, kind=kind, want_each=False)
    assert torch.equal(total, alone)
    assert flags == 0
    assert close(float(total[0]), want, NORM_TOL)
    assert close(float(total[1]), min(1.0, 0.5 / (want + 1e-6)), FACTOR_TOL)
    for got, w in zip(each.tolist(), want_each):
        assert close(got, w, NORM_TOL)


def test_no_tensors():
    h = nshb.tensors([])
    ws = nshb.tensor_workspace(h)
    total = torch.full((2,), -1.0, device=DEV)
    nshb.grad_norm(h, total, ws, max_norm=2.0)
    assert total.tolist() == [0.0, 1.0] and nshb.device_status(ws) == 0
    nshb.clip_grads(h, 2.0, total.fill_(-1), ws)
    assert total.tolist() == [0.0, 1.0]
    nshb.scale_grads(h, total)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [1, 3, 8, 15])
def test_any_alignment_and_leading_dimension(dtype, offset):
    base = make([(300 * 1000 + 64,)], dtype, seed=offset)[0]
    flat = base[offset:offset + 9001]
    wide = base[offset:offset + 290 * 1000].view(290, 1000)[:, 13:700]     # long rows, each its own alignment
    thin = base[offset:offset + 290 * 1000].view(290, 1000)[:, 5:42]       # short rows
    one = base[offset:offset + 100 * 1000].view(100, 1000)[:, 7:8]          # a column
    ts = [flat, wide, thin, one]
    want, want_each = exact_norms(ts)
    total, each, _ = norm(ts)
    assert close(float(total[0]), want, NORM_TOL)
    for got, w in zip(each.tolist(), want_each):
        assert close(got, w, NORM_TOL)


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 1e25, 3e37])
def test_squares_outside_fp32(scale):
    # 1e-42 is below the smallest normal fp32; the largest sum of squares here is near 1e81
    ts = make([(5000,), (70, 3)], torch.float32, seed=1, scale=scale)
    ts.append(torch.zeros(100, device=DEV))
    want, _ = exact_norms(ts)
    total, each, flags = norm(ts)
    # a subnormal result is off by half a subnormal step
    step = 2.0 ** -149 if want < 2.0 ** -126 else 0.0
    expected = want if want < 3.4e38 else math.inf
    assert float(total[0]) == expected or abs(float(total[0]) - want) <= NORM_TOL * want + step / 2
    assert flags == (nshb.NSHB_DEV_NONFINITE if expected == math.inf else 0)


@pytest.mark.parametrize("kind", [nshb.NSHB_NORM_L2, nshb.NSHB_NORM_INF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(kind, dtype, bad):
    ts = make([(3000,), (40, 50)], dtype)
    ts[1][39, 49] = bad
    total, each, flags = norm(ts, kind=kind)
    assert flags == nshb.NSHB_DEV_NONFINITE
    if math.isnan(bad):
        assert math.isnan(total[0]) and math.isnan(total[1]) and math.isnan(each[1])
    else:
        assert float(total[0]) == math.inf and float(total[1]) == 0.0 and float(each[1]) == math.inf
    assert math.isfinite(each[0])
    h = nshb.tensors(ts)
    ws = nshb.tensor_workspace(h)
    nshb.grad_norm(h, total, ws)                       # no limit: the same
    assert math.isnan(total[1]) if math.isnan(bad) else float(total[1]) == 0.0
    ts[1][39, 49] = 0
    nshb.grad_norm(h, total, ws)                       # the flag is of the last call
    assert nshb.device_status(ws) == 0 and float(total[1]) == 1.0


@pytest.mark.parametrize("src_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dst_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("count", [0, 1, 800])
@pytest.mark.parametrize("offset", [0, 1, 5, 8])
def test_clip_into(src_dtype, dst_dtype, count, offset):
    shapes = [(33, 65), (1, 5000), (700, 301) if count else (70, 31)] + [(1, 3)] * count
    src = make(shapes, src_dtype, seed=count)
    lds = [c + (9 if i == 2 else 0) for i, (_, c) in enumerate(shapes)]
    size = sum(r * ld for (r, _), ld in zip(shapes, lds))
    buf = torch.full((size + offset,), 7.0, device=DEV, dtype=dst_dtype)
    keep = torch.ones_like(buf, dtype=torch.bool)
    dst, at = [], offset
    for (r, c), ld in zip(shapes, lds):
        dst.append(buf[at:at + r * ld].view(r, ld)[:, :c])
        keep[at:at + r * ld].view(r, ld)[:, :c] = False
        at += r * ld
    before = [s.clone() for s in src]
    hs, hd = nshb.tensors(src), nshb.tensors(dst)
    ws = nshb.tensor_workspace(hs).fill_(0xAB)
    total = torch.zeros(2, device=DEV)
    nshb.clip_grads(hs, 0.125, total, ws, dst=hd)
    plain, _, _ = norm(src, max_norm=0.125, want_each=False)
    assert torch.equal(total, plain) and float(total[1]) < 1
    for s, b, d in zip(src, before, dst):
        assert torch.equal(s, b)
        assert torch.equal(d, (b.float() * total[1]).to(dst_dtype))
    assert bool((buf[keep] == 7.0).all())      # nothing between the rows or before the first is written


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("max_norm", [0.25, 1e9])
@pytest.mark.parametrize("kind", [nshb.NSHB_NORM_L2, nshb.NSHB_NORM_INF])
def test_clip_in_place(dtype, max_norm, kind):
    ts = make([(513, 255), (77,), (2000,)], dtype, seed=3)
    before = [t.clone() for t in ts]
    h = nshb.tensors(ts)
    ws = nshb.tensor_workspace(h)
    total = torch.zeros(2, device=DEV)
    nshb.clip_grads(h, max_norm, total, ws, kind=kind)
    want, _ = exact_norms(before, kind)
    assert close(float(total[1]), min(1.0, max_norm / (want + 1e-6)), FACTOR_TOL)
    for t, b in zip(ts, before):
        assert torch.equal(t, (b.float() * total[1]).to(dtype))
    if max_norm < want:
        after, _ = exact_norms(ts, kind)
        # each element rounded by at most half a step
        assert after <= max_norm * (1 + FACTOR_TOL + torch.finfo(dtype).eps / 2)


def test_scale_by_a_factor_on_the_device():
    ts = make([(100, 30), (5,)], torch.float32, seed=9)
    want = [t * 0.3 for t in ts]
    nshb.scale_grads(nshb.tensors(ts), torch.tensor([0.3], device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(ts, want))


def test_a_stream_and_a_captured_graph():
    ts = make([(1000, 999), (64,), (2048, 2048)], torch.bfloat16, seed=4)
    out = [torch.zeros_like(t) for t in ts]
    h, d = nshb.tensors(ts), nshb.tensors(out)
    ws, total = nshb.tensor_workspace(h), torch.zeros(2, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nshb.clip_grads(h, 0.5, total, ws, dst=d)
    for seed in (5, 6):
        for t, n in zip(ts, make([t.shape for t in ts], torch.bfloat16, seed=seed)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = total.clone(), [o.clone() for o in out]
        with torch.cuda.stream(side):
            nshb.clip_grads(h, 0.5, total, ws, dst=d)
        side.synchronize()
        assert torch.equal(total, got[0]) and all(torch.equal(a, b) for a, b in zip(out, got[1]))


def test_a_run_of_more_than_two_to_the_31_elements():
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[0], t[-1], t[1 << 31] = 3.0, 4.0, 12.0
    total, _, _ = norm([t], max_norm=6.5)
    assert float(total[0]) == 13.0
    h = nshb.tensors([t])
    nshb.clip_grads(h, 6.5, total, nshb.tensor_workspace(h))
    assert [float(t[i]) for i in (0, -1, 1 << 31)] == [1.5, 2.0, 6.0]
