"""Products of 4-bit matrices against fp64 products of the values that the codes stand for.

Bound.  Code x code is a multiple of 1/4 up to 36, a block's scale product multiplies it; the
accumulator is fp32.  Whatever the order, every partial sum is at most S = sum |a||b| of the element,
and each of the K/64 accumulation steps may round (or truncate) once at S's magnitude, the sum inside a
step being at least as wide: |error| <= (K/64 + 8 joins of parts + 2 global scales) 2^-23 S, plus half a step of
D's type.
"""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = nshb.NSHB_MXFP4, nshb.NSHB_NVFP4


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def operand(rows, cols, fmt, seed, spread=1.0):
    """(Fp4 on the device, its values in fp64), from random codes and scales."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    blocks = -(-cols // ref.BLOCK[fmt])
    if fmt == MX:
        byte = np.clip(127 + np.round(rng.standard_normal((rows, blocks)) * 3 * spread), 1, 250).astype(np.uint8)
    else:
        byte = rng.integers(0, 127, (rows, blocks)).astype(np.uint8)
    g = float(np.float32(rng.uniform(0.01, 3))) if fmt == NV else 1.0
    q = nshb.Fp4(rows, cols, fmt, torch.from_numpy(ref.pack(code).reshape(-1).copy()).to(DEV),
                 torch.from_numpy(ref.tile_scales(byte, rows, cols, fmt)).to(DEV),
                 torch.tensor([g], device=DEV) if fmt == NV else None)
    return q, ref.values(code, byte, g, fmt)


def check(d, a, b, k):
    """d (any stride) against a b^T within the bound above."""
    got = d.detach().double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (k / 64 + 10) * 2.0 ** -23 * size + torch.finfo(d.dtype).eps / 2 * np.abs(want) * 1.01
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    off = np.abs(got - want)[~nan] - tol[~nan]
    assert (off <= 0).all(), (off.max(), np.argwhere((np.abs(got - want) > tol))[:5])


def product(ops_a, ops_b, dtype, lds=None):
    ds, bufs = [], []
    for i, a in enumerate(ops_a):
        n = (ops_b or ops_a)[i].rows
        pad = lds[i] if lds else 0
        buf = torch.full((a.rows + 2, n + pad + 3), 7.0, dtype=dtype, device=DEV)
        flat = torch.full((a.rows * (n + pad) + 64,), 7.0, dtype=dtype, device=DEV)
        ds.append(flat[:a.rows * (n + pad)].view(a.rows, n + pad)[:, :n] if pad == 0 else buf[1:1 + a.rows, 1:1 + n])
        bufs.append((buf, flat))
    hd = nshb.tensors(ds)
    ws = nshb.tensor_workspace(hd).fill_(0xAB)
    nshb.fp4_matmul(nshb.fp4_matrices(ops_a), nshb.fp4_matrices(ops_b) if ops_b else None, hd, ws)
    assert nshb.device_status(ws) == 0
    for d, (buf, flat) in zip(ds, bufs):     # nothing outside the result is written
        d_copy = d.clone()
        d.fill_(7.0)
        assert bool((buf == 7.0).all()) and bool((flat == 7.0).all())
        d.copy_(d_copy)
    return ds


SIZES = [(1, 1, 1), (1, 128, 64), (128, 128, 64), (128, 128, 128), (128, 128, 256), (128, 128, 1024), (1, 16, 31),
         (3, 5, 17), (1, 300, 2048), (16, 257, 300), (17, 129, 512), (33, 1000, 640), (64, 640, 2049), (65, 66, 67),
         (300, 1, 700), (300, 40, 130), (1, 2000, 4096), (2, 130, 6200), (20, 500, 5000), (64, 256, 8192), (130, 140, 8192),
         (200, 300, 4100), (1100, 500, 8192), (257, 7, 6145), (129, 255, 257), (256, 384, 511), (1000, 777, 1333), (130, 2000, 96)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_products(fmt, dtype, size):
    m, n, k = size
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    for pad in (0, 5):
        check(product([a], [b], dtype, [pad])[0], av, bv, k)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("size", [(1, 1), (40, 100), (128, 300), (129, 64), (400, 1000), (768, 2000), (300, 8200),
                                  (500, 4097)])
def test_gram(fmt, size):
    d, k = size
    a, av = operand(d, k, fmt, 3)
    out = product([a], None, torch.float32)[0]
    check(out, av, av, k)
    assert torch.equal(out, out.t())


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(2304, 2304, 64), (2300, 2310, 256), (4100, 1300, 1000), (1300, 4100, 1537), (19000, 200, 333)])
def test_products_of_many_tiles(fmt, dtype, size):
    test_products(fmt, dtype, size)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("d,k", [(3000, 700), (3333, 256)])
def test_gram_of_many_tiles(fmt, d, k):
    test_gram(fmt, (d, k))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_a_list_of_many_tiles(fmt):
    shapes = [(1500, 700, 300), (257, 300, 4000), (5, 600, 100), (1000, 1000, 70), (300, 300, 0), (1500, 900, 513)] * 2
    a = [operand(m, k, fmt, 10 + i) for i, (m, n, k) in enumerate(shapes)]
    b = [operand(n, k, fmt, 90 + i) for i, (m, n, k) in enumerate(shapes)]
    ds = product([x[0] for x in a], [x[0] for x in b], torch.float32)
    for d, x, y, (m, n, k) in zip(ds, a, b, shapes):
        check(d, x[1], y[1], k)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_a_list(fmt):
    shapes = [(5, 300, 70), (7, 200, 500), (0, 4, 64), (300, 300, 64), (3, 4, 0), (1, 2, 3), (200, 0, 9), (150, 150, 300)] * 7
    a = [operand(m, k, fmt, 10 + i) for i, (m, n, k) in enumerate(shapes)]
    b = [operand(n, k, fmt, 90 + i) for i, (m, n, k) in enumerate(shapes)]
    ds = product([x[0] for x in a], [x[0] for x in b], torch.float32)
    for d, x, y, (m, n, k) in zip(ds, a, b, shapes):
        if m and n:
            check(d, x[1], y[1], k)
    x, xv = operand(9, 0, fmt, 5)
    out = product([x], None, torch.bfloat16)[0]
    assert bool((out == 0).all())


@pytest.mark.parametrize("gram", [False, True])
def test_shapes_and_formats_in_turn(gram):
    """More products of one kind than a launch takes, others between them, both formats and result types."""
    shapes = ([(130, 140, 64)] * 5 + [(1, 200, 300), (40, 130, 5000), (700, 800, 256), (0, 9, 70), (300, 310, 8200)]) * 11
    fmts = [MX if i % 3 else NV for i in range(len(shapes))]
    a = [operand(m, k, f, 10 + i) for i, ((m, n, k), f) in enumerate(zip(shapes, fmts))]
    b = a if gram else [operand(n, k, f, 500 + i) for i, ((m, n, k), f) in enumerate(zip(shapes, fmts))]
    for dtype in (torch.float32, torch.bfloat16):
        ds = product([x[0] for x in a], None if gram else [x[0] for x in b], dtype)
        for d, x, y, (m, n, k) in zip(ds, a, b, shapes):
            if m:
                check(d, x[1], y[1], k)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("m", [2, 200])
def test_nan_blocks_reach_their_row_and_no_other(fmt, m):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(m, 333, generator=g)
    w = torch.randn(300, 333, generator=g)
    x[1, 40], w[7, 100], w[299, 332] = float("nan"), float("inf"), -float("inf")
    ops, vals = [], []
    for t in (x, w):
        q = nshb.fp4_empty(*t.shape, fmt, DEV)
        ht = nshb.tensors([t.to(DEV)])
        nshb.fp4_quantize(ht, nshb.fp4_matrices([q]), nshb.tensor_workspace(ht))
        ops.append(q)
        vals.append(ref.values(*ref.quantize(t.double().numpy(), fmt), fmt))
    out = product([ops[0]], [ops[1]], torch.float32)[0]
    check(out, vals[0], vals[1], 333)
    assert int(torch.isnan(out).sum()) == 300 + 2 * (m - 1)


def test_the_same_bits_again_on_a_stream_and_in_a_graph():
    a, _ = operand(3, 2048, NV, 1)
    b, _ = operand(1000, 2048, NV, 2)
    d = torch.empty(3, 1000, device=DEV)
    ha, hb, hd = nshb.fp4_matrices([a]), nshb.fp4_matrices([b]), nshb.tensors([d])
    ws = nshb.tensor_workspace(hd)
    nshb.fp4_matmul(ha, hb, hd, ws)
    want = d.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nshb.fp4_matmul(ha, hb, hd, ws)
    for _ in range(3):
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)
    d.zero_()
    side.wait_stream(torch.cuda.current_stream())
    nshb.fp4_matmul(ha, hb, hd, ws, stream=side)
    side.synchronize()
    assert torch.equal(d, want)
