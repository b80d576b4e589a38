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
