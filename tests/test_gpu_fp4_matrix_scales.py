"""Matrix scales (NVFP4's *global) over fp32's whole range: products of which only the product of the two scales leaves
it, and values under scales that are no power of two.

The fp32 accumulator is exact up to (K/64 + 8) 2^-23 of the summed magnitudes (see test_gpu_fp4_matmul.py); the
scales add two roundings, and a result below the smallest normal number is off by half a subnormal step more, in
fp32 (2^-150) and then in D's type.
"""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NV = nshb.NSHB_NVFP4


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def operand(rows, cols, g, seed):
    """(Fp4 with the matrix scale g and a first row of zero codes, its codes' and scales' values in fp64 without g)."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    code[0] = 0
    byte = rng.integers(8, 127, (rows, -(-cols // 16))).astype(np.uint8)
    q = nshb.Fp4(rows, cols, NV, torch.from_numpy(ref.pack(code).reshape(-1).copy()).to(DEV),
                 torch.from_numpy(ref.tile_scales(byte, rows, cols, NV)).to(DEV),
                 torch.tensor([g], dtype=torch.float32, device=DEV))
    return q, ref.values(code, byte, 1.0, NV)


# one operand's scale and the other's: both tiny, both huge, one of each, subnormal ones, zero, no powers of two
PAIRS = [(2.0 ** -77, 2.0 ** -77), (1e-20, 3e-19), (2.0 ** 70, 2.0 ** 70), (2.0 ** 117, 2.0 ** -126), (2.0 ** 100, 2.0 ** 20),
         (1e-40, 3e5), (3e5, 1e-40), (2.0 ** -126, 2.0 ** -20), (0.0, 1e38), (0.37, 0.011), (2.0 ** -64, 2.0 ** -60)]
# one row (D transposed), few rows, a split sum of either kind, 64-wide and 128-wide tiles, CTA pairs
SIZES = [(1, 300, 200), (20, 90, 500), (40, 100, 6200), (130, 140, 8200), (300, 200, 333), (2400, 2600, 256)]


def compare(d, v, w, g, h, k):
    gg, hh = np.float64(np.float32(g)), np.float64(np.float32(h))
    got = d.double().cpu().numpy()
    want, size = (v @ w.T) * gg * hh, (np.abs(v) @ np.abs(w).T) * (abs(gg) * abs(hh))
    info = torch.finfo(d.dtype)
    tol = (k / 64 + 10) * 2.0 ** -23 * size + info.eps / 2 * np.abs(want) * 1.01 + info.smallest_normal * info.eps / 2 + 2.0 ** -150
    assert not np.isnan(got).any()
    over = np.abs(want) - tol > info.max * (1 + info.eps / 4)
    assert (got[over] == np.copysign(np.inf, want[over])).all()
    near = ~over & (np.abs(want) + tol >= info.max)
    off = np.abs(got - want)[~over & ~near] - tol[~over & ~near]
    assert (off <= 0).all(), (g, h, off.max())
    return int(over.sum())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_products(size, dtype):
    m, n, k = size
    for i, (g, h) in enumerate(PAIRS):
        (a, v), (b, w) = operand(m, k, g, 2 * i), operand(n, k, h, 2 * i + 1)
        d = torch.full((m, n), 7.0, dtype=dtype, device=DEV)
        hd = nshb.tensors([d])
        ws = nshb.tensor_workspace(hd)
        nshb.fp4_matmul(nshb.fp4_matrices([a]), nshb.fp4_matrices([b]), hd, ws)
        assert nshb.device_status(ws) == 0
        compare(d, v, w, g, h, k)
        assert bool((d[0] == 0).all()) and bool((d[:, 0] == 0).all())


@pytest.mark.parametrize("size", [(100, 500), (300, 8200), (2600, 256)])
def test_gram(size):
    d, k = size
    for i, g in enumerate((2.0 ** -70, 2.0 ** 70, 1e-25, 5e18, 0.37)):
        a, v = operand(d, k, g, i)
        out = torch.full((d, d), 7.0, device=DEV)
        hd = nshb.tensors([out])
        ws = nshb.tensor_workspace(hd)
        nshb.fp4_matmul(nshb.fp4_matrices([a]), None, hd, ws)
        assert nshb.device_status(ws) == 0
        compare(out, v, v, g, g, k)
        assert torch.equal(out, out.t()) and bool((out[0] == 0).all())
