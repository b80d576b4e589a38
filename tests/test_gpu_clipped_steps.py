"""Steps on clipped gradients: the factor read by the momentum pass (nshb_step_scaled), and a data-parallel
optimizer with max_grad_norm.

The scaled step is the step on factor * G without a rounding of the product.  For fp32 gradients that is the
step on the tensors that nshb_scale_grads leaves, bit for bit.  For bf16 ones it is the oracle's step on the fp64
product, within the bounds the unscaled steps are held to (O 2e-2, M 1e-6 plus one rounding of the product, 2^-24).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import newton_schulz_hyperball_b200 as nshb  # noqa: E402
from gpu_harness import GpuSet, rel_fro  # noqa: E402
from newton_schulz_hyperball_b200 import sharding  # noqa: E402
from newton_schulz_hyperball_b200 import workloads as wl  # noqa: E402
from oracle import nshb_oracle as o  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
OPS = {"muon": nshb.NSHB_OP_MUON, "hyperball": nshb.NSHB_OP_HYPERBALL, "radial_brake": nshb.NSHB_OP_RADIAL_BRAKE,
       "himuon": nshb.NSHB_OP_HIMUON, "relative_update": nshb.NSHB_OP_RELATIVE_UPDATE}
SHAPES = [(256, 512), (512, 256), (200, 330), (5, 7), (40, 1)]


def state(dtype, seed=3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    W = [(0.02 * torch.randn(s, device=DEV, generator=g)).to(dtype) for s in SHAPES]
    G = [torch.randn(s, device=DEV, generator=g).to(dtype) for s in SHAPES]
    M = [0.1 * torch.randn(s, device=DEV, generator=g) for s in SHAPES]
    return W, G, M


def params(kind, f32):
    kw = dict(tile=128) if kind == "himuon" else {}
    return nshb.params(ns_precision=nshb.NSHB_F32 if f32 and kind != "himuon" else nshb.NSHB_BF16, **kw)


@pytest.mark.parametrize("kind", list(OPS))
@pytest.mark.parametrize("factor", [1.0, 0.3, 0.0])
def test_fp32_gradients_give_the_bits_of_scaling_first(kind, factor):
    f = torch.tensor([factor], device=DEV)
    got = []
    for fused in (True, False):
        W, G, M = state(torch.float32)
        mats, p = nshb.matrices(W, G, M), params(kind, True)
        ws = nshb.workspace(mats, p, OPS[kind])
        if fused:
            nshb.step_scaled(OPS[kind], mats, p, f, ws)
        else:
            nshb.scale_grads(nshb.tensors(G), f)
            getattr(nshb, kind + "_step")(mats, p, ws)
        nshb.device_status(ws)
        got.append((W, M))
    for a, b in zip(got[0][0] + got[0][1], got[1][0] + got[1][1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", list(OPS))
def test_a_factor_of_one_is_the_step(kind):
    got = []
    for fused in (True, False):
        W, G, M = state(torch.bfloat16)
        mats, p = nshb.matrices(W, G, M), params(kind, False)
        ws = nshb.workspace(mats, p, OPS[kind])
        if fused:
            nshb.step_scaled(OPS[kind], mats, p, torch.ones(1, device=DEV), ws)
        else:
            getattr(nshb, kind + "_step")(mats, p, ws)
        assert nshb.device_status(ws) == 0
        got.append((W, M))
    for a, b in zip(got[0][0] + got[0][1], got[1][0] + got[1][1]):
        assert torch.equal(a, b)


def test_clipped_bf16_step_follows_the_oracle():
    shapes = [(256, 512), (384, 128)]
    Ws = [wl.init_weight(5, i, r, c, bf16=True).astype(np.float64) for i, (r, c) in enumerate(shapes)]
    Gs = [wl.gradient(5, i, 0, r, c, bf16=True).astype(np.float64) for i, (r, c) in enumerate(shapes)]
    gs = GpuSet(Ws, bf16=True)
    gs.set_grads(Gs)
    g = nshb.tensors(gs.G)
    total = torch.zeros(2, device=DEV)
    nshb.grad_norm(g, total, nshb.tensor_workspace(g), max_norm=0.05)
    norm = float(np.sqrt(sum((x ** 2).sum() for x in Gs)))
    factor = min(1.0, 0.05 / (norm + 1e-6))
    assert factor < 1 and abs(float(total[1]) - factor) <= 5 * 2.0 ** -24 * factor
    p = nshb.params(eta=0.02)
    ws = nshb.workspace(gs.mats, p, nshb.NSHB_OP_HYPERBALL)
    nshb.step_scaled(nshb.NSHB_OP_HYPERBALL, gs.mats, p, total[1:], ws)
    assert nshb.device_status(ws) == 0
    _, Mg, Og = gs.host()
    for i in range(len(shapes)):
        _, Mr, Or, _ = o.hyperball_step(Ws[i], factor * Gs[i], np.zeros_like(Ws[i]), eta=0.02, rho=None)
        assert rel_fro(Mg[i], Mr) <= 1e-6 + 6 * 2.0 ** -24
        assert rel_fro(Og[i], Or) <= 2e-2


def test_norm_and_clipped_step_in_one_graph():
    def run(graphed):
        W, G, M = state(torch.bfloat16)
        mats, p = nshb.matrices(W, G, M), params("hyperball", False)
        ws = nshb.workspace(mats, p, nshb.NSHB_OP_HYPERBALL)
        g, total = nshb.tensors(G), torch.zeros(2, device=DEV)
        gws = nshb.tensor_workspace(g)

        def step():
            nshb.grad_norm(g, total, gws, max_norm=0.5)
            nshb.step_scaled(nshb.NSHB_OP_HYPERBALL, mats, p, total[1:], ws)
        if graphed:
            graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(graph, stream=side):
                step()
            step = graph.replay
        for k in range(3):
            for x in G:
                x.mul_(0.5)
            step()
        torch.cuda.synchronize()
        return W + M + [total]
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_sharded_optimizer_clips():
    shapes = [(256, 256), (300, 200), (64, 512)]
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    W = [(0.02 * torch.randn(s, device=DEV, generator=g)).bfloat16() for s in shapes]
    G = [torch.randn(s, device=DEV, generator=g).bfloat16() for s in shapes]
    rho = torch.stack([w.float().norm() for w in W])
    Wa = [w.clone() for w in W]
    opt = sharding.ShardedOptimizer(Wa, rho, sharding.make_plan(shapes, 1, 0), "hyperball", eta=0.02, max_grad_norm=1.0)
    opt.step(G)
    assert opt.device_status() == 0
    Wb, M = [w.clone() for w in W], [torch.zeros(s, device=DEV) for s in shapes]
    mats, p = nshb.matrices(Wb, G, M), nshb.params(eta=0.02, rho=rho)
    t, total = nshb.tensors(G), torch.zeros(2, device=DEV)
    nshb.grad_norm(t, total, nshb.tensor_workspace(t), max_norm=1.0)
    ws = nshb.workspace(mats, p, nshb.NSHB_OP_HYPERBALL)
    nshb.step_scaled(nshb.NSHB_OP_HYPERBALL, mats, p, total[1:], ws)
    assert torch.equal(opt.grad_total, total) and float(total[1]) < 1
    assert torch.equal(sharding.clip_factor(total[:1], 1.0), total[1:])
    for a, b in zip(Wa, Wb):
        assert torch.equal(a, b)
