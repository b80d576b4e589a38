"""Several clipped steps of ShardedOptimizer over gloo ranks on CPU, with ranks that own nothing.

The library's calls are stood in for by their definitions in fp32 and fp64 (the kernels have their GPU tests); the
plan, the exchange of gradients, the norm over the ranks, its factor and the exchange of weights are the module's own."""
import os
import socket

import pytest
import torch
import torch.multiprocessing as mp

from newton_schulz_hyperball_b200 import sharding

MAX_NORM = 0.75
LR = 0.5


def _free_port():
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    p = s.getsockname()[1]
    s.close()
    return p


def stand_in(nshb):
    """A step is W <- W - LR factor G."""
    def grad_norm(g, total, ws, max_norm):
        n = sum(t.double().square().sum() for t in g).sqrt().float()
        total.copy_(torch.stack((n, (torch.full_like(n, max_norm) / (n + 1e-6)).clamp(max=1.0))))

    def step_scaled(op, mats, p, factor, ws, stream=None):
        for w, g, _ in mats:
            w.sub_(LR * factor * g)
    nshb.tensors = list
    nshb.tensor_workspace = lambda g: None
    nshb.params = lambda **kw: None
    nshb.matrices = lambda W, G, M: list(zip(W, G, M))
    nshb.workspace = lambda *a, **k: None
    nshb.grad_norm, nshb.step_scaled = grad_norm, step_scaled


def gradient(rank, step, i, shape):
    g = torch.Generator().manual_seed(1000 * rank + 10 * step + i)
    return torch.randint(-8, 9, shape, generator=g).float()       # whole numbers: the sum over ranks is exact


def _worker(rank, world, port, shapes, steps, out_dir):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    import torch.distributed as dist
    from datetime import timedelta
    import newton_schulz_hyperball_b200 as nshb
    stand_in(nshb)
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        W = [torch.ones(s) for s in shapes]
        opt = sharding.ShardedOptimizer(W, torch.ones(len(shapes)), sharding.make_plan(shapes, world, rank), "muon",
                                        average=False, max_grad_norm=MAX_NORM)
        totals = []
        for step in range(steps):
            opt.step([gradient(rank, step, i, s) for i, s in enumerate(shapes)])
            totals.append(opt.grad_total.clone())
        torch.save((totals, W), os.path.join(out_dir, f"r{rank}.pt"))
        dist.barrier()
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("world,shapes", [
    (2, [(6, 5), (4, 4), (3, 7)]),
    (3, [(6, 5)]),                  # two ranks own nothing
    (3, [(6, 5), (4, 4)]),          # one does
])
def test_every_step_clips_by_its_own_norm(tmp_path, world, shapes):
    steps = 4
    mp.start_processes(_worker, args=(world, _free_port(), shapes, steps, str(tmp_path)), nprocs=world,
                       start_method="spawn", join=True)
    got = [torch.load(tmp_path / f"r{r}.pt") for r in range(world)]
    W = [torch.ones(s, dtype=torch.float64) for s in shapes]
    half = 2.0 ** -24
    for step in range(steps):
        G = [sum(gradient(r, step, i, s).double() for r in range(world)) for i, s in enumerate(shapes)]
        norm = float(sum(g.square().sum() for g in G).sqrt())
        factor = min(1.0, MAX_NORM / (norm + 1e-6))
        assert factor < 1
        for totals, _ in got:
            # each rank's norm and the norm over the ranks are rounded once, the factor's sum and quotient too
            assert abs(float(totals[step][0]) - norm) <= 2 * half * norm, step
            assert abs(float(totals[step][1]) - factor) <= 4 * half * factor, step
        for w, g in zip(W, G):
            w.sub_(LR * factor * g)
    for totals, weights in got:
        for t, u in zip(totals, got[0][0]):
            assert torch.equal(t, u)
        for w, v in zip(weights, W):
            # a step's term is at most LR MAX_NORM, off by the factor's 4 roundings and 2 of its own; the difference is
            # rounded at a size of at most 1 + steps LR MAX_NORM
            term = LR * MAX_NORM
            assert float((w.double() - v).abs().max()) <= steps * half * (6 * term + 1 + steps * term)
