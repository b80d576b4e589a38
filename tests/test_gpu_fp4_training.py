"""4-bit layer inputs in the Newton-Muon step, and the operators around a step used one after the other.

The 4-bit step is held to the oracle's on the values that the codes stand for, with the bounds of the bf16 step.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import newton_schulz_hyperball_b200 as nshb  # noqa: E402
from gpu_harness import GpuSet, rel_fro  # noqa: E402
from newton_schulz_hyperball_b200 import workloads as wl  # noqa: E402
from oracle import nshb_oracle as o  # noqa: E402
from tests import fp4_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [nshb.NSHB_MXFP4, nshb.NSHB_NVFP4]


def quantized(x, fmt, transpose=False):
    r, c = (x.shape[1], x.shape[0]) if transpose else x.shape
    q = nshb.fp4_empty(r, c, fmt, DEV)
    h = nshb.tensors([x])
    nshb.fp4_quantize(h, nshb.fp4_matrices([q]), nshb.tensor_workspace(h), transpose=transpose)
    return q


@pytest.mark.parametrize("fmt", FORMATS)
def test_newton_step_with_4_bit_inputs_follows_the_oracle(fmt):
    # inputs of different widths and lengths: padded, one and several diagonal blocks, odd lengths
    z_shape = [(320, 1000), (64, 257), (576, 4096)]
    shapes, z_index = [(200, 320), (320, 320), (700, 64), (64, 576), (600, 576)], [0, 0, 1, 2, 2]
    Zs = [wl.layer_input(9, j, d, n).astype(np.float64) for j, (d, n) in enumerate(z_shape)]
    # the forward pass holds tokens x features
    qs = [quantized(torch.from_numpy(z.T.copy()).to(DEV).bfloat16(), fmt, transpose=True) for z in Zs]
    Zv = [ref.values(*ref.quantize(z, fmt), fmt) for z in Zs]
    Ws = [wl.init_weight(9, i, r, c, bf16=True).astype(np.float64) for i, (r, c) in enumerate(shapes)]
    Gs = [wl.gradient(9, i, 0, r, c, bf16=True).astype(np.float64) for i, (r, c) in enumerate(shapes)]
    gs = GpuSet(Ws, bf16=True)
    for i, z in enumerate(z_index):
        gs.mats[i].z_index = z
    gs.set_grads(Gs)
    p = nshb.params(eta=0.02, ridge_rel=1e-3)
    ws = nshb.workspace(gs.mats, p, nshb.NSHB_OP_NEWTON_MUON, z_rows=[d for d, _ in z_shape], n_tokens=64).fill_(0xAB)
    nshb.newton_muon_step_fp4(gs.mats, nshb.fp4_matrices(qs), p, ws)
    assert nshb.device_status(ws) == 0
    _, Mg, Og = gs.host()
    for i, z in enumerate(z_index):
        _, Mr, Or, _ = o.newton_muon_step(Ws[i], Gs[i], np.zeros_like(Ws[i]), Zv[z], ridge_rel=1e-3, eta=0.02, rho=None)
        assert rel_fro(Mg[i], Mr) <= 1e-6, i
        assert rel_fro(Og[i], Or) <= 2e-2, (i, rel_fro(Og[i], Or))


def test_4_bit_and_bf16_inputs_of_the_same_values_agree():
    """MX values are bf16 numbers: both steps get the same Z, and differ by the Gram's summation alone."""
    d, n = 512, 2048
    q = quantized(torch.from_numpy(wl.layer_input(4, 0, d, n)).to(DEV).bfloat16(), nshb.NSHB_MXFP4)
    Z = torch.empty(d, n, dtype=torch.bfloat16, device=DEV)
    nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([Z]))
    W0, G0 = wl.init_weight(4, 0, 256, d, bf16=True), wl.gradient(4, 0, 0, 256, d, bf16=True)
    out = []
    for four in (True, False):
        gs = GpuSet([W0], bf16=True)
        gs.mats[0].z_index = 0
        gs.set_grads([G0])
        p = nshb.params(eta=0.02)
        ws = nshb.workspace(gs.mats, p, nshb.NSHB_OP_NEWTON_MUON, z_rows=[d], n_tokens=n)
        if four:
            nshb.newton_muon_step_fp4(gs.mats, nshb.fp4_matrices([q]), p, ws)
        else:
            nshb.newton_muon_step(gs.mats, [Z], n, p, ws)
        assert nshb.device_status(ws) == 0
        out.append(gs.host()[2][0])
    # each side is within 1e-2 of the fp64 map on such inputs
    assert rel_fro(out[0], out[1]) <= 2e-2


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 333])
def test_a_training_step_with_the_operators_around_it(fmt, tokens):
    """Activations to 4 bits, product with 4-bit weights, clipped gradients, Newton-Muon step on the 4-bit
    inputs, the new weights and their transposes to 4 bits, product for the activations' gradient."""
    d_in, d_out = 320, 192
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    x = torch.randn(tokens, d_in, device=DEV, generator=g).bfloat16()
    W = (0.05 * torch.randn(d_out, d_in, device=DEV, generator=g)).bfloat16()
    dy = torch.randn(tokens, d_out, device=DEV, generator=g).bfloat16()

    def values(q):
        v = torch.empty(q.rows, q.cols, device=DEV)
        nshb.fp4_dequantize(nshb.fp4_matrices([q]), nshb.tensors([v]))
        return v.double()

    def product(a, b, dtype=torch.float32):
        d = torch.empty(a.rows, b.rows, dtype=dtype, device=DEV)
        h = nshb.tensors([d])
        ws = nshb.tensor_workspace(h)
        nshb.fp4_matmul(nshb.fp4_matrices([a]), nshb.fp4_matrices([b]), h, ws)
        assert nshb.device_status(ws) == 0
        k = a.cols
        size = values(a).abs() @ values(b).abs().t()
        assert bool(((d.double() - values(a) @ values(b).t()).abs() <= (k / 64 + 10) * 2.0 ** -23 * size).all())
        return d

    y = product(quantized(x, fmt), quantized(W, fmt))
    assert y.shape == (tokens, d_out)
    G = (dy.float().t() @ x.float()).bfloat16()
    t, total = nshb.tensors([G]), torch.zeros(2, device=DEV)
    nshb.clip_grads(t, 1.0, total, nshb.tensor_workspace(t))
    assert float(G.double().norm()) <= 1 + 2.0 ** -8 + 1e-5
    z = quantized(x, fmt, transpose=True)
    M = torch.zeros(d_out, d_in, device=DEV)
    W0 = W.double().cpu().numpy()
    mats = nshb.matrices([W], [G], [M], z_index=[0])
    p = nshb.params(eta=0.02, ridge_rel=1e-1)
    ws = nshb.workspace(mats, p, nshb.NSHB_OP_NEWTON_MUON, z_rows=[d_in], n_tokens=64)
    nshb.newton_muon_step_fp4(mats, nshb.fp4_matrices([z]), p, ws)
    assert nshb.device_status(ws) == 0
    assert abs(float(W.double().norm()) - np.linalg.norm(W0)) <= 1e-3 * np.linalg.norm(W0)
    dx = product(quantized(dy, fmt), quantized(W, fmt, transpose=True))
    assert dx.shape == (tokens, d_in)
