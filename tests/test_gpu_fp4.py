"""4-bit quantisation and values against the plain fp64 form: equal bits everywhere (the format's
rounding is exact, see nshb_fp4 in include/nshb.h)."""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [nshb.NSHB_MXFP4, nshb.NSHB_NVFP4]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def matrix(rows, cols, dtype, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    return x.to(dtype)


def quantize(xs, fmt, transpose=False, stream=None):
    qs = []
    for x in xs:
        r, c = (x.shape[1], x.shape[0]) if transpose else x.shape
        q = nshb.fp4_empty(r, c, fmt, DEV)
        q.codes.fill_(0xEE)
        q.scales.fill_(0xEE)
        qs.append(q)
    hx, hq = nshb.tensors(xs), nshb.fp4_matrices(qs)
    ws = nshb.tensor_workspace(hx).fill_(0xAB) if fmt == nshb.NSHB_NVFP4 else None
    nshb.fp4_quantize(hx, hq, ws, transpose=transpose, stream=stream)
    return qs


def check(x, q, fmt, transpose=False):
    h = x.detach().cpu().double().numpy()
    h = h.T if transpose else h
    code, byte, g = ref.quantize(h, fmt)
    got = q.codes.cpu().numpy().reshape(q.rows, -1)
    assert np.array_equal(got, ref.pack(code))
    assert np.array_equal(q.scales.cpu().numpy(), ref.tile_scales(byte, q.rows, q.cols, fmt))
    if fmt == nshb.NSHB_NVFP4:
        assert float(q.global_scale) == g
    want = ref.values(code, byte, g, fmt)
    for dtype in DTYPES:
        out = torch.full((q.rows, q.cols), 9.0, dtype=dtype, device=DEV)
        nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([out]))
        assert np.array_equal(out.cpu().double().numpy(), torch.from_numpy(want.copy()).to(dtype).double().numpy(), equal_nan=True)


SIZES = [(1, 1), (1, 16), (3, 17), (1, 31), (2, 32), (5, 33), (127, 128), (128, 127), (129, 129), (64, 300), (300, 64),
         (257, 1000), (1000, 257), (1, 4000), (4000, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(fmt, dtype, transpose, size):
    x = matrix(*size, dtype, seed=sum(size)).to(DEV)
    check(x, quantize([x], fmt, transpose)[0], fmt, transpose)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transpose", [False, True])
def test_borders_between_codes(fmt, dtype, transpose):
    """Values on the border of two codes and the nearest fp32 (or bf16) values to both sides of it."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    rows = []
    for s in [1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875]:
        m = torch.tensor(np.concatenate([mids, -mids]) * s, dtype=dtype)
        bits = m.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        for d in (-2, -1, 0, 1, 2):
            v = (bits + d).view(dtype).float()
            for top in (6.0 * s, 4.0):
                # blocks of 32 whose largest value fixes the scale
                rows.append(torch.cat([torch.tensor([top]), v[:15], torch.tensor([top]), v[3:18]]))
    x = torch.stack(rows).to(dtype)
    x = torch.cat([x, x * 2.0 ** -9, x * 2.0 ** 30])
    x = torch.cat([x, torch.full((x.shape[0], 32), 448.0 * 6, dtype=dtype)], dim=1) if fmt == nshb.NSHB_NVFP4 else x
    x = (x.t() if transpose else x).contiguous().to(DEV)
    check(x, quantize([x], fmt, transpose)[0], fmt, transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_every_bf16_value_under_every_scale(transpose):
    """NVFP4 with a matrix scale of 1: all bf16 values from an eighth of each scale to six times it, and each
    bf16 value as the largest of its block."""
    mantissas = torch.arange(128, 256, dtype=torch.float64) / 128
    every = torch.cat([mantissas * 2.0 ** e for e in range(-13, 12)])
    scales = [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1] + [m * 2.0 ** -9 for m in range(1, 8)]
    blocks = []
    for s in scales:
        v = every[(every >= s / 8) & (every <= 6 * s)]
        v = torch.cat([v, v.new_zeros(-len(v) % 15)]).view(-1, 15) * torch.tensor([1.0, -1.0] * 7 + [1.0], dtype=v.dtype)
        blocks.append(torch.cat([v.new_full((len(v), 1), 6 * s), v], dim=1))
    tops = every[every <= 2688]
    blocks.append(torch.cat([tops[:, None], tops.new_zeros(len(tops), 15)], dim=1))
    b = torch.cat(blocks)
    x = torch.cat([b, b.new_zeros(-len(b) % 16, 16)]).view(-1, 256)
    x[0, 0] = 2688.0
    assert torch.equal(x, x.bfloat16().double())
    x = (x.t() if transpose else x).contiguous().to(torch.bfloat16).to(DEV)
    check(x, quantize([x], nshb.NSHB_NVFP4, transpose)[0], nshb.NSHB_NVFP4, transpose)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-39, 1e-37, 1e-30, 1.0, 1e30, 3e38])
def test_the_whole_range_of_the_exponent(fmt, dtype, transpose, scale):
    x = matrix(70, 100, torch.float32, seed=3, spread=0.5).double()
    x = (x / x.abs().max() * scale).to(dtype).to(DEV)
    check(x, quantize([x], fmt, transpose)[0], fmt, transpose)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
def test_more_tiles_than_the_gpu_takes_at_once(fmt, transpose):
    xs = [matrix(r, c, torch.bfloat16, seed=r).to(DEV) for r, c in ((1500, 3000), (130, 1290), (2000, 2600))]
    for x, q in zip(xs, quantize(xs, fmt, transpose)):
        check(x, q, fmt, transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_dtypes_and_formats_in_one_list(transpose):
    kinds = [(d, f) for d in DTYPES for f in FORMATS] * 2
    xs = [matrix(40 + 7 * i, 90 - 5 * i, d, seed=i).to(DEV) for i, (d, _) in enumerate(kinds)]
    qs = [nshb.fp4_empty(*(x.shape[::-1] if transpose else x.shape), f, DEV) for x, (_, f) in zip(xs, kinds)]
    h = nshb.tensors(xs)
    nshb.fp4_quantize(h, nshb.fp4_matrices(qs), nshb.tensor_workspace(h), transpose=transpose)
    outs = [torch.empty(q.rows, q.cols, dtype=d, device=DEV) for q, (d, _) in zip(qs, kinds[::-1])]
    nshb.fp4_dequantize(nshb.fp4_matrices(qs), nshb.tensors(outs))
    for x, q, o, (_, f) in zip(xs, qs, outs, kinds):
        check(x, q, f, transpose)
        one = torch.empty_like(o)
        nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([one]))
        assert torch.equal(o, one)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transpose", [False, True])
def test_not_finite_and_zero(fmt, dtype, transpose):
    x = matrix(200, 160, dtype, seed=5)
    x[0] = 0
    x[1, :40] = -0.0
    x[3, 5], x[77, 130], x[150, 31] = float("nan"), float("inf"), -float("inf")
    x[:, 9] = 0
    x = x.to(DEV)
    check(x, quantize([x], fmt, transpose)[0], fmt, transpose)
    z = torch.zeros(40, 50, dtype=dtype, device=DEV)
    check(z, quantize([z], fmt, transpose)[0], fmt, transpose)
    n = torch.full((40, 50), float("nan"), dtype=dtype, device=DEV)
    check(n, quantize([n], fmt, transpose)[0], fmt, transpose)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
def test_a_list_with_strides_offsets_and_empty_ones(fmt, transpose):
    base = matrix(300, 400, torch.bfloat16, seed=7).to(DEV)
    f32 = matrix(90, 70, torch.float32, seed=8).to(DEV)
    xs = [base[:, 3:200], base[17:18, :], torch.zeros(0, 5, device=DEV), base[:, 16:144], f32, f32[:, 1:2],
          torch.zeros(4, 0, device=DEV)]
    for x, q in zip(xs, quantize(xs, fmt, transpose)):
        if x.numel():
            check(x, q, fmt, transpose)
    many = [base[i:i + 1, :33] for i in range(250)]             # more than one launch
    for x, q in list(zip(many, quantize(many, fmt, transpose)))[::83]:
        check(x, q, fmt, transpose)


def test_values_keep_to_their_rows():
    q = quantize([matrix(37, 45, torch.float32).to(DEV)], nshb.NSHB_MXFP4)[0]
    out = torch.full((40, 64), 5.0, device=DEV)
    nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([out[1:38, 8:53]]))
    rest = out.clone()
    rest[1:38, 8:53] = 5.0
    assert bool((rest == 5.0).all()) and not bool((out[1:38, 8:53] == 5.0).all())


def test_stream_and_graph():
    x = matrix(256, 512, torch.bfloat16).to(DEV)
    q = nshb.fp4_empty(256, 512, nshb.NSHB_NVFP4, DEV)
    hx, hq = nshb.tensors([x]), nshb.fp4_matrices([q])
    ws = nshb.tensor_workspace(hx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nshb.fp4_quantize(hx, hq, ws)
    x.copy_(matrix(256, 512, torch.bfloat16, seed=11))
    graph.replay()
    torch.cuda.synchronize()
    check(x, q, nshb.NSHB_NVFP4)
