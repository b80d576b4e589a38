"""The clip factor of a norm formed over ranks (sharding.clip_factor): one sum and one quotient in fp32, each rounded
once, so the bits that nshb_grad_norm writes next to the same norm."""
import numpy as np
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb
from newton_schulz_hyperball_b200 import sharding

MAX_NORMS = [0.3, 1.0, 2.7, 1e-3, 1e30, float("inf")]


@pytest.mark.parametrize("max_norm", MAX_NORMS)
def test_one_rounding_each(max_norm):
    g = torch.Generator().manual_seed(1)
    norm = torch.cat([torch.exp(8 * torch.randn(5000, generator=g)), torch.tensor([0.0, 1e-45, 1e-20, max_norm, 3e38])])
    norm = norm[torch.isfinite(norm)]
    want = np.minimum(np.float32(max_norm) / (norm.numpy() + np.float32(1e-6)), np.float32(1))
    got = sharding.clip_factor(norm, max_norm)
    assert got.dtype == torch.float32 and np.array_equal(got.numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("max_norm", MAX_NORMS)
def test_the_librarys_bits(max_norm):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    t = torch.zeros(1, device="cuda")
    h = nshb.tensors([t])
    ws, total = nshb.tensor_workspace(h), torch.zeros(2, device="cuda")
    g = torch.Generator().manual_seed(2)
    for v in torch.exp(4 * torch.randn(200, generator=g)).tolist() + [0.0, 1e-45, 3e38, float("inf"), float("nan")]:
        t.fill_(v)
        nshb.grad_norm(h, total, ws, max_norm=max_norm)
        f = sharding.clip_factor(total[:1], max_norm)
        assert torch.equal(f, total[1:]) or (bool(torch.isnan(f)) and bool(torch.isnan(total[1]))), (v, f, total)
