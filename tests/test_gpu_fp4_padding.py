"""Scale bytes past a 4-bit matrix's rows, in its last tile of 128, are nobody's: any byte there, NaN's among them, leaves
every result's bits as they are."""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from newton_schulz_hyperball_b200 import workloads as wl
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [nshb.NSHB_MXFP4, nshb.NSHB_NVFP4]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def quantized(x, fmt):
    q = nshb.fp4_empty(*x.shape, fmt, DEV)
    h = nshb.tensors([x])
    nshb.fp4_quantize(h, nshb.fp4_matrices([q]), nshb.tensor_workspace(h))
    return q


def with_padding(q, byte):
    """The same matrix with `byte` for every scale past its rows."""
    blocks = -(-q.cols // 128) * 128 // ref.BLOCK[q.format]
    live = ref.tile_scales(np.ones((q.rows, blocks), dtype=np.uint8), q.rows, blocks * ref.BLOCK[q.format], q.format)
    s = q.scales.clone()
    s[torch.from_numpy(live == 0).to(DEV)] = byte
    return nshb.Fp4(q.rows, q.cols, q.format, q.codes, s, q.global_scale)


def nan_byte(fmt):
    return 0xFF if fmt == nshb.NSHB_MXFP4 else 0x7F


def product(a, b, m, n):
    d = torch.full((m, n), 3.0, device=DEV)
    h = nshb.tensors([d])
    ws = nshb.tensor_workspace(h)
    nshb.fp4_matmul(nshb.fp4_matrices([a]), nshb.fp4_matrices([b]) if b else None, h, ws)
    assert nshb.device_status(ws) == 0
    return d


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [(1, 200, 300), (20, 90, 500), (40, 100, 6200), (130, 140, 8200), (300, 200, 333), (2401, 2500, 256)])
def test_products_and_values(fmt, size):
    m, n, k = size
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    a, b = (quantized(torch.randn(r, k, device=DEV, generator=g), fmt) for r in (m, n))
    want, gram = product(a, b, m, n), product(b, None, n, n)
    assert not bool(torch.isnan(want).any())
    for byte in (nan_byte(fmt), 0x55):
        a2, b2 = with_padding(a, byte), with_padding(b, byte)
        assert n % 128 == 0 or not torch.equal(b2.scales, b.scales)
        assert torch.equal(product(a2, b2, m, n), want) and torch.equal(product(b2, None, n, n), gram)
        values = [torch.empty(n, k, device=DEV) for _ in range(2)]
        nshb.fp4_dequantize(nshb.fp4_matrices([b, b2]), nshb.tensors(values))
        assert torch.equal(*values)


@pytest.mark.parametrize("fmt", FORMATS)
def test_newton_step(fmt):
    rows = [64, 320, 576]
    Z = [quantized(torch.from_numpy(wl.layer_input(9, j, d, 700)).to(DEV).bfloat16(), fmt) for j, d in enumerate(rows)]
    outs = []
    for qs in (Z, [with_padding(q, nan_byte(fmt)) for q in Z]):
        W = [torch.from_numpy(wl.init_weight(9, i, 200, d, bf16=True)).to(DEV).bfloat16() for i, d in enumerate(rows)]
        G = [torch.from_numpy(wl.gradient(9, i, 0, 200, d, bf16=True)).to(DEV).bfloat16() for i, d in enumerate(rows)]
        M = [torch.zeros(200, d, device=DEV) for d in rows]
        mats, p = nshb.matrices(W, G, M, z_index=[0, 1, 2]), nshb.params(eta=0.02)
        ws = nshb.workspace(mats, p, nshb.NSHB_OP_NEWTON_MUON, z_rows=rows, n_tokens=64).fill_(0xAB)
        nshb.newton_muon_step_fp4(mats, nshb.fp4_matrices(qs), p, ws)
        assert nshb.device_status(ws) == 0
        outs.append(W)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
