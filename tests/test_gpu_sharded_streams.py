"""ShardedOptimizer.step on a stream of its own: after the gradients that the current stream still computes, and
before what the current stream does with the weights."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from newton_schulz_hyperball_b200 import sharding  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [(256, 256), (300, 200), (64, 512)]


@pytest.mark.parametrize("max_grad_norm", [None, 1.0])
@pytest.mark.parametrize("how", ["stream", "pointer", "default"])
def test_a_step_on_a_side_stream_waits_for_the_gradients_and_is_waited_for(max_grad_norm, how):
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    W = [(0.02 * torch.randn(s, device=DEV, generator=g)).bfloat16() for s in SHAPES]
    G = [torch.randn(s, device=DEV, generator=g).bfloat16() for s in SHAPES]
    rho = torch.stack([w.float().norm() for w in W])
    opts = [sharding.ShardedOptimizer([w.clone() for w in W], rho, sharding.make_plan(SHAPES, 1, 0), "hyperball",
                                      eta=0.02, max_grad_norm=max_grad_norm) for _ in range(2)]
    for _ in range(2):
        opts[0].step(G)
    torch.cuda.synchronize()
    late = [torch.zeros_like(x) for x in G]
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(mine):
        for _ in range(2):
            for x in late:
                x.zero_()
            torch.cuda._sleep(50_000_000)       # the gradients come some 25 ms after the call
            for x, y in zip(late, G):
                x.copy_(y)
            opts[1].step(late, {"stream": side, "pointer": side.cuda_stream, "default": 0}[how])
            seen = [w.clone() for w in opts[1].W]
    mine.synchronize()
    assert opts[1].device_status() == 0
    for a, b, c in zip(opts[0].W, opts[1].W, seen):
        assert torch.equal(a, b) and torch.equal(a, c)
    if max_grad_norm is not None:
        assert torch.equal(opts[0].grad_total, opts[1].grad_total) and float(opts[0].grad_total[1]) < 1
