"""Where ShardedOptimizer.step puts its work when it is given a stream (CPU, streams stood in for by names).

Every part has to be on that stream, after the caller's stream (which holds the gradients) and before what the caller
does next (which reads the weights)."""
import contextlib

import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from newton_schulz_hyperball_b200 import sharding


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.device = name, log, torch.device("cpu")

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")


@pytest.fixture
def log(monkeypatch):
    log, at = [], []
    at.append(Stream("caller", log))

    @contextlib.contextmanager
    def on(stream):
        at.append(stream or at[-1])
        yield
        at.pop()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream("default", log))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda pointer, device=None: Stream(f"at {pointer}", log))
    monkeypatch.setattr(torch.cuda, "stream", on)

    def part(name, where=lambda *a, **k: at[-1]):
        return lambda *a, **k: log.append(f"{name} on {where(*a, **k).name}")
    given = lambda *a, **k: (a[-1] if isinstance(a[-1], Stream) else k.get("stream")) or at[-1]  # noqa: E731
    monkeypatch.setattr(sharding, "reduce_scatter_grads", part("reduce"))
    monkeypatch.setattr(sharding, "all_gather_weights", part("gather"))
    monkeypatch.setattr(nshb, "grad_norm", part("norm"))
    monkeypatch.setattr(nshb, "step_scaled", part("step", given))
    monkeypatch.setattr(nshb, "muon_step", part("step", given))
    for name in ("tensors", "tensor_workspace", "params", "matrices", "workspace"):
        monkeypatch.setattr(nshb, name, lambda *a, **k: object())
    return log


def step(log, stream, max_grad_norm):
    W = [torch.ones(2, 3)]
    opt = sharding.ShardedOptimizer(W, torch.ones(1), sharding.make_plan([(2, 3)], 1, 0), "muon", max_grad_norm=max_grad_norm)
    opt.step([torch.ones(2, 3)], stream)
    return log


@pytest.mark.parametrize("max_grad_norm", [None, 1.0])
@pytest.mark.parametrize("stream", ["side", 0, 77])
def test_all_of_a_step_is_on_its_stream(log, max_grad_norm, stream):
    name = {"side": "side", 0: "default", 77: "at 77"}[stream]
    got = step(log, Stream("side", log) if stream == "side" else stream, max_grad_norm)
    parts = ["reduce"] + (["norm"] if max_grad_norm else []) + ["step", "gather"]
    assert [x for x in got if " on " in x] == [f"{p} on {name}" for p in parts]
    assert got.index(f"{name} waits for caller") < got.index(f"reduce on {name}")
    assert len(got) - 1 - got[::-1].index(f"caller waits for {name}") > got.index(f"gather on {name}")


@pytest.mark.parametrize("max_grad_norm", [None, 1.0])
def test_without_one_it_is_on_the_callers(log, max_grad_norm):
    got = step(log, None, max_grad_norm)
    assert got == ["reduce on caller"] + (["norm on caller"] if max_grad_norm else []) + ["step on caller", "gather on caller"]
