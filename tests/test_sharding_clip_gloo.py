"""The gradient norm over ranks on CPU: every rank passes the norm of the gradients it owns, all get the norm of all
of them (gloo, spawned processes), and the factor that nshb_grad_norm forms from a norm."""
import math
import os
import socket

import torch
import torch.multiprocessing as mp

from newton_schulz_hyperball_b200 import sharding


def _free_port():
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    p = s.getsockname()[1]
    s.close()
    return p


def _worker(rank, world, port, norms, out_dir):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    import torch.distributed as dist
    from datetime import timedelta
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        got = [sharding.global_grad_norm(torch.tensor([n[rank]])) for n in norms]
        torch.save(torch.cat(got), os.path.join(out_dir, f"n{rank}.pt"))
        dist.barrier()
    finally:
        dist.destroy_process_group()


def test_ranks_agree_on_the_norm(tmp_path):
    # a rank that owns nothing passes 0; norms whose squares leave fp32
    norms = [(3.0, 4.0, 0.0), (1e30, 2e30, 2e30), (1e-30, 0.0, 0.0), (math.inf, 1.0, 0.0), (math.nan, 1.0, 2.0)]
    mp.start_processes(_worker, args=(3, _free_port(), norms, str(tmp_path)), nprocs=3, start_method="spawn", join=True)
    got = [torch.load(tmp_path / f"n{r}.pt") for r in range(3)]
    want = torch.tensor([5.0, 3e30, 1e-30, math.inf, math.nan])
    for g in got:
        assert torch.equal(torch.isnan(g), torch.isnan(want))
        # inputs rounded to fp32, result rounded once
        assert bool(((g[:3] - want[:3]).abs() <= 2 * 2.0 ** -24 * want[:3]).all()) and g[3] == math.inf


def test_clip_factor():
    f = sharding.clip_factor(torch.tensor([0.5, 2.0, 0.0, math.inf, math.nan]), 1.0)
    assert f[0] == 1 and f[2] == 1 and f[3] == 0 and math.isnan(f[4])
    assert abs(float(f[1]) - 1 / (2 + 1e-6)) <= 2 * 2.0 ** -24
