"""The README's Python examples run as they stand, and the clipping one clips what it shows by one norm."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_examples():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    steps, rest = blocks[:2], blocks[2:]
    ns = {}
    for b in steps:
        exec(b, ns)
    biases = [torch.randn(768, device="cuda"), torch.randn(77, device="cuda").bfloat16()]
    ns["biases_grads"] = [b.clone() for b in biases]
    norm = sum(float(t.double().square().sum()) for t in ns["G"] + biases) ** 0.5
    for b in rest:
        exec(b, ns)
    torch.cuda.synchronize()
    nshb, total = ns["nshb"], ns["total"]
    for ws in ("ws", "gws", "ws_n", "ws_z"):
        assert nshb.device_status(ns[ws]) == 0, ws
    # three roundings of the norm, two more of the factor (see test_gpu_grad_norm.py)
    assert abs(float(total[0]) - norm) <= 3 * 2.0 ** -24 * norm
    factor = 1 / (norm + 1e-6)
    assert abs(float(total[1]) - factor) <= 5 * 2.0 ** -24 * factor
    for got, b in zip(ns["biases_grads"], biases):
        assert torch.equal(got, (b.float() * total[1]).to(b.dtype))
