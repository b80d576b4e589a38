"""Both triangles of a Gram matrix: every element stored, (i, j) with the bits of (j, i), the same on every call, for D
of either type, aligned to 16 bytes or not.  Bound of an element: see test_gpu_fp4_matmul.py."""
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from tests.test_gpu_fp4_matmul import check, operand

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [nshb.NSHB_MXFP4, nshb.NSHB_NVFP4]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# around the 32, 64, 128 and 256 rows of blocks and tiles; sums shared by a cluster; CTA pairs
SIZES = [(1, 64), (31, 100), (32, 64), (33, 64), (63, 300), (64, 64), (65, 1000), (127, 70), (128, 8200), (129, 64), (130, 4100),
         (255, 8200), (257, 256), (300, 5000), (1000, 300), (2560, 64), (2601, 300)]


def gram(ops, ds):
    h = nshb.tensors(ds)
    ws = nshb.tensor_workspace(h).fill_(0xAB)
    nshb.fp4_matmul(nshb.fp4_matrices(ops), None, h, ws)
    assert nshb.device_status(ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_each_element_once(fmt, dtype, size):
    d, k = size
    a, v = operand(d, k, fmt, d + k)
    first = None
    for pad, offset in ((0, 0), (8, 0), (3, 1)):
        buf = torch.full((d + 1, d + pad), float("nan"), dtype=dtype, device=DEV)
        out = buf.view(-1)[offset:offset + d * (d + pad)].view(d, d + pad)[:, :d]
        for _ in range(2):
            out.fill_(float("nan"))
            gram([a], [out])
            assert torch.equal(out, out.t())             # no NaN is left either
            first = out.clone() if first is None else first
            assert torch.equal(out, first)
        rest = buf.clone()
        rest.view(-1)[offset:offset + d * (d + pad)].view(d, d + pad)[:, :d] = float("nan")
        assert bool(torch.isnan(rest).all())             # nothing else is written
    check(first, v, v, k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_in_a_list(fmt):
    ops = [operand(d, k, fmt, i) for i, (d, k) in enumerate(SIZES)]
    ds = [torch.full((q.rows, q.rows), float("nan"), device=DEV) for q, _ in ops]
    gram([q for q, _ in ops], ds)
    for (q, v), d in zip(ops, ds):
        assert torch.equal(d, d.t())
        check(d, v, v, q.cols)
