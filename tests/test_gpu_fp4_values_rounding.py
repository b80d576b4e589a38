"""Values of NVFP4 matrices whose scale is no power of two: code x scale x *global rounded once, also to bf16, where a
rounding to fp32 before it would decide half of the ties wrongly.  Equal bits."""
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


def to_bf16(v):
    """The nearest bf16 value of each fp64 one, ties to even, without a step in between."""
    step = 2.0 ** np.maximum(np.frexp(v)[1] - 8, -133).astype(np.float64)
    r = np.rint(v / step) * step
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, v), r)


def every_code_and_scale(negative_first):
    """One row: blocks of all 16 codes under each E4M3 scale."""
    code = np.tile(np.arange(16, dtype=np.uint8), 127)
    if negative_first:
        code = (code + 8) % 16
    return code[None, :], np.arange(127, dtype=np.uint8)[None, :]


def near_ties():
    """Scales g for which some code x scale, times g, is within half an fp32 unit of the middle of two bf16 values
    without being there: a g = T (1 + d), |d| < 2^-24, T with nine bits."""
    out = []
    for a in (1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875, 2.0625, 2.8125):
        for t in range(257, 512, 30):
            g = np.float32(t / a)
            if np.float64(a) * np.float64(g) != t and np.float32(a * np.float64(g)) == t:
                out.append(float(g))
    return out


def test_the_cases_are_what_they_are_for():
    """Enough of the scales below round wrongly through fp32."""
    code, byte = every_code_and_scale(False)
    wrong = 0
    for g in near_ties():
        v = ref.values(code, byte, g, NV)
        with np.errstate(invalid="ignore"):
            through = to_bf16(v.astype(np.float32).astype(np.float64))
        wrong += int((through != to_bf16(v))[~np.isnan(v)].sum())
    assert wrong > 50


SCALES = [0.37, -1.7, 3e5, 1e-37, 1e-40, 2.0 ** -149, 3 * 2.0 ** -149, 1.3e35, 1.1e38, 3.4e38, 2.0 ** -126, 2.0 ** 117, 0.0]


@pytest.mark.parametrize("part", range(4))
def test_one_rounding(part):
    for i, g in enumerate((near_ties() + SCALES + [2.0 ** -100 * x for x in near_ties()[:20]]
                           + [2.0 ** -138 * x for x in near_ties()[:20]])[part::4]):
        code, byte = every_code_and_scale(i % 2 == 1)
        rows = 1 + 130 * (i % 3 == 0)
        code, byte = np.repeat(code, rows, 0), np.repeat(byte, rows, 0)
        cols = code.shape[1]
        g = float(np.float32(g))
        q = nshb.Fp4(rows, cols, NV, torch.from_numpy(ref.pack(code).reshape(-1).copy()).to(DEV),
                     torch.from_numpy(ref.tile_scales(byte, rows, cols, NV)).to(DEV),
                     torch.tensor([g], dtype=torch.float64).float().to(DEV))
        want = ref.values(code, byte, g, NV)
        for pad in (0, 1):          # whole rows of 16-byte stores, and element by element
            b = torch.empty(rows, cols + pad, dtype=torch.bfloat16, device=DEV)[:, :cols]
            f = torch.empty(rows, cols + pad, dtype=torch.float32, device=DEV)[:, :cols]
            h = nshb.fp4_matrices([q])
            nshb.fp4_dequantize(h, nshb.tensors([b]))
            nshb.fp4_dequantize(h, nshb.tensors([f]))
            with np.errstate(over="ignore"):
                assert np.array_equal(f.cpu().numpy(), want.astype(np.float32)), g
            assert np.array_equal(b.cpu().double().numpy(), to_bf16(want)), g
