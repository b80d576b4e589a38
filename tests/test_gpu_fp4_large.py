"""4-bit matrices and results of more than 2^31 elements: the last rows and columns as exact as the first ones (parts
compared with the plain fp64 form; bounds of the products: see test_gpu_fp4_matmul.py)."""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [nshb.NSHB_MXFP4, nshb.NSHB_NVFP4]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
def test_quantisation_and_values(fmt, transpose):
    rows, cols = 33000, 66000                                  # 2.18e9 elements; values and codes pass 2^31 and 2^30
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    spots = [(slice(0, 5), slice(0, 600)), (slice(rows - 37, rows), slice(cols - 700, cols)), (slice(16000, 16002), slice(0, cols))]
    for r, c in spots:
        x[r, c] = torch.randn(x[r, c].shape, device=DEV, generator=g).bfloat16()
    x[rows - 1, cols - 1] = 2000.0                             # decides the matrix scale
    q = nshb.fp4_empty(*((cols, rows) if transpose else (rows, cols)), fmt, DEV)
    h = nshb.tensors([x])
    nshb.fp4_quantize(h, nshb.fp4_matrices([q]), nshb.tensor_workspace(h), transpose=transpose)
    v = torch.empty(q.rows, q.cols, dtype=torch.bfloat16, device=DEV)
    nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([v]))
    v = v.t() if transpose else v
    for r, c in spots:
        # whole blocks along the 4-bit matrix's columns, and the element that decides the scale in one more row
        b0 = (r.start if transpose else c.start) // 32 * 32
        part = x[b0:r.stop, c] if transpose else x[r, b0:c.stop]
        part = part.double().cpu().numpy().T if transpose else part.double().cpu().numpy()
        code, byte, whole = ref.quantize(np.vstack([part, np.full((1, part.shape[1]), 2000.0)]), fmt)
        want = ref.values(code, byte, whole, fmt)[:-1, (r.start if transpose else c.start) - b0:]
        want = torch.from_numpy((want.T if transpose else want).copy()).to(torch.bfloat16)
        assert torch.equal(v[r, c].cpu(), want)
    assert int((v != 0).sum()) <= sum((r.stop - r.start) * (c.stop - c.start) for r, c in spots)


@pytest.mark.parametrize("gram", [False, True])
def test_a_result(gram):
    m, n, k = (47000, 47000, 96) if gram else (70001, 33000, 96)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    ops, vals = [], []
    for rows in (m,) if gram else (m, n):
        x = torch.randn(rows, k, device=DEV, generator=g)
        q = nshb.fp4_empty(rows, k, nshb.NSHB_NVFP4, DEV)
        h = nshb.tensors([x])
        nshb.fp4_quantize(h, nshb.fp4_matrices([q]), nshb.tensor_workspace(h))
        nshb.fp4_dequantize(nshb.fp4_matrices([q]), h)
        ops.append(nshb.fp4_matrices([q]))
        vals.append(x.double())
    a, b = vals[0], vals[-1]
    d = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    hd = nshb.tensors([d])
    ws = nshb.tensor_workspace(hd)
    nshb.fp4_matmul(ops[0], None if gram else ops[1], hd, ws)
    assert nshb.device_status(ws) == 0
    assert not any(bool(torch.isnan(d[i:i + 5000]).any()) for i in range(0, m, 5000))
    for r, c in ((slice(0, 300), slice(0, 300)), (slice(m - 300, m), slice(n - 300, n)), (slice(m - 300, m), slice(0, 300)),
                 (slice(0, 300), slice(n - 300, n)), (slice(m // 2, m // 2 + 3), slice(0, n))):
        want, size = a[r] @ b[c].t(), a[r].abs() @ b[c].abs().t()
        tol = (k / 64 + 10) * 2.0 ** -23 * size + torch.finfo(torch.bfloat16).eps / 2 * want.abs() * 1.01
        assert bool(((d[r, c].double() - want).abs() <= tol).all())
