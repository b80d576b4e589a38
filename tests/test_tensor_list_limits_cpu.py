"""Limits of the entry points on lists of tensors: what the header allows is not refused, and what it does not is refused
before anything is queued (CPU only)."""
import ctypes

import pytest

import newton_schulz_hyperball_b200 as nshb

TOTAL, WS = 0x7000000, 0x8000000


def fake(*shapes, dtype=nshb.NSHB_BF16, base=0x10000000):
    arr = (nshb.nshb_tensor * len(shapes))()
    for i, (r, c, ld) in enumerate(shapes):
        arr[i].rows, arr[i].cols, arr[i].ld, arr[i].dtype, arr[i].data = r, c, ld, dtype, base + 0x1000000 * i
    return arr


def size(t):
    out = ctypes.c_size_t(0)
    return nshb.lib().nshb_tensor_workspace_size(t, len(t), ctypes.byref(out))


@pytest.mark.parametrize("ld", [-1, 0, 3, (1 << 40) + 1, (1 << 63) - 1, -(1 << 63)])
@pytest.mark.parametrize("rows", [0, 1])
def test_the_leading_dimension_of_one_row_is_not_looked_at(rows, ld):
    assert size(fake((5, 7, 7), (rows, 5, ld))) == nshb.NSHB_OK


BIG = (1 << 30) + 1


def test_rows_apart_from_one_another_have_a_limit_and_it_is_met_before_any_launch():
    small, big = (5, 7, 7), (BIG, 1, 2)
    lib = nshb.lib()
    t, good = fake(*[small] * 600, big), fake(*[small] * 600, (BIG, 1, 1), base=1 << 40)   # the big one in a second launch
    n = len(t)
    assert size(t) == nshb.NSHB_ERR_UNSUPPORTED and size(good) == nshb.NSHB_OK
    assert lib.nshb_grad_norm(t, n, 0, 1.0, TOTAL, None, WS, 1 << 20, None) == nshb.NSHB_ERR_UNSUPPORTED
    for args in ((t, None), (t, good), (good, t)):
        assert lib.nshb_clip_grads(*args, n, 0, 1.0, TOTAL, WS, 1 << 20, None) == nshb.NSHB_ERR_UNSUPPORTED
        assert lib.nshb_scale_grads(*args, n, TOTAL, None) == nshb.NSHB_ERR_UNSUPPORTED
    assert size(fake((1 << 30, 1, 2))) == size(fake((1 << 40, 1, 1))) == nshb.NSHB_OK


def test_a_quantisation_of_more_than_one_launchs_windows_is_not_refused():
    """65 strided sources of 2^24 rows: more than 2^30 pieces for the pass that finds the largest magnitudes."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up: only where nothing can be launched")
    n = 65
    x = fake(*[(1 << 24, 256, 257)] * n)
    q = (nshb.nshb_fp4 * n)()
    for i in range(n):
        q[i].rows, q[i].cols, q[i].format = 1 << 24, 256, nshb.NSHB_NVFP4
        q[i].codes, q[i].scales, q[i].global_ = 0x40000000, 0x50000000, 0x60000000
    assert nshb.lib().nshb_fp4_quantize(x, q, n, 0, WS, 1 << 20, None) == nshb.NSHB_ERR_CUDA    # no GPU to launch on
