"""step_scaled without a factor is refused like every missing pointer (CPU only)."""
import pytest
import torch

import newton_schulz_hyperball_b200 as nshb


@pytest.mark.parametrize("kept", [False, True])
def test_a_missing_factor(kept):
    m = (nshb.nshb_matrix * 1)()
    m[0].rows = m[0].cols = m[0].ld = 64
    m[0].W, m[0].G, m[0].M = 0x1000000, 0x2000000, 0x3000000
    if kept:
        m._keep = ([torch.zeros(64, 64)],)      # as matrices() leaves it
    with pytest.raises(nshb.NshbError) as e:
        nshb.step_scaled(nshb.NSHB_OP_MUON, m, nshb.params(), None, (0x9000000, 1 << 30), stream=0)
    assert e.value.status == nshb.NSHB_ERR_NULL
