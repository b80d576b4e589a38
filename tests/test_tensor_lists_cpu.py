"""Refusals of the entry points on lists of tensors: returned before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

import newton_schulz_hyperball_b200 as nshb

TOTAL = 0x7000000
WS = 0x8000000


def fake(*shapes, dtype=nshb.NSHB_BF16, base=0x10000000):
    arr = (nshb.nshb_tensor * max(len(shapes), 1))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols, arr[i].ld, arr[i].dtype = r, c, c, dtype
        arr[i].data = base + 0x1000000 * i
    arr._n = len(shapes)
    return arr


def size(t, n=None):
    out = ctypes.c_size_t(0)
    return nshb.lib().nshb_tensor_workspace_size(t, t._n if n is None else n, ctypes.byref(out)), out.value


def norm(t, kind=0, max_norm=1.0, total=TOTAL, each=None, ws=WS, ws_bytes=1 << 20, n=None):
    return nshb.lib().nshb_grad_norm(t, t._n if n is None else n, kind, max_norm, total, each, ws, ws_bytes, None)


def clip(s, d=None, kind=0, max_norm=1.0, total=TOTAL, ws=WS, ws_bytes=1 << 20):
    return nshb.lib().nshb_clip_grads(s, d, s._n, kind, max_norm, total, ws, ws_bytes, None)


def test_struct_layout():
    assert ctypes.sizeof(nshb.nshb_tensor) == 40 and nshb.nshb_tensor.data.offset == 32


def test_workspace_grows_with_the_number_of_tensors_alone():
    few, many = size(fake((2, 3)))[1], size(fake(*[(2, 3)] * 300))[1]
    assert 256 < few < many <= size(fake(*[(20000, 30000)] * 300))[1] == many
    assert many % 256 == 0 and size(fake())[0] == nshb.NSHB_OK


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), nshb.NSHB_ERR_SHAPE),
    (dict(cols=-1), nshb.NSHB_ERR_SHAPE),
    (dict(ld=4), nshb.NSHB_ERR_SHAPE),
    (dict(data=0x10000001), nshb.NSHB_ERR_SHAPE),
    (dict(rows=(1 << 40) + 1), nshb.NSHB_ERR_UNSUPPORTED),
    (dict(rows=1 << 21, cols=1 << 20, ld=1 << 20), nshb.NSHB_ERR_UNSUPPORTED),
    (dict(ld=(1 << 40) + 1), nshb.NSHB_ERR_UNSUPPORTED),
    (dict(dtype=2), nshb.NSHB_ERR_DTYPE),
    (dict(reserved=1), nshb.NSHB_ERR_PARAM),
    (dict(data=None), nshb.NSHB_ERR_NULL),
])
def test_a_bad_tensor_is_refused_everywhere(change, code):
    t = fake((3, 5), (2, 5), (4, 5))
    for k, v in change.items():
        setattr(t[1], k, v)
    good = fake((3, 5), (2, 5), (4, 5), base=0x20000000)
    assert size(t)[0] == norm(t) == clip(t) == clip(good, t) == code
    assert nshb.lib().nshb_scale_grads(t, None, 3, TOTAL, None) == code
    assert nshb.lib().nshb_scale_grads(good, t, 3, TOTAL, None) == code


def test_bad_arguments():
    t = fake((3, 5))
    assert norm(t, n=-1) == size(t, -1)[0] == nshb.NSHB_ERR_SHAPE
    assert norm(t, total=None) == clip(t, total=None) == norm(t, ws=None) == nshb.NSHB_ERR_NULL
    assert nshb.lib().nshb_grad_norm(None, 1, 0, 1.0, TOTAL, None, WS, 1 << 20, None) == nshb.NSHB_ERR_NULL
    assert nshb.lib().nshb_tensor_workspace_size(t, 1, None) == nshb.NSHB_ERR_NULL
    assert nshb.lib().nshb_scale_grads(t, None, 1, None, None) == nshb.NSHB_ERR_NULL
    assert nshb.lib().nshb_scale_grads(t, None, 1, TOTAL + 2, None) == nshb.NSHB_ERR_SHAPE
    assert norm(t, total=TOTAL + 2) == norm(t, each=TOTAL + 1) == nshb.NSHB_ERR_SHAPE
    for bad in (0.0, -1.0, float("nan")):
        assert norm(t, max_norm=bad) == clip(t, max_norm=bad) == nshb.NSHB_ERR_PARAM
    assert norm(t, kind=2) == clip(t, kind=-1) == nshb.NSHB_ERR_PARAM
    need = size(t)[1]
    assert norm(t, ws_bytes=need - 1) == clip(t, ws_bytes=need - 1) == norm(t, ws=WS + 128) == nshb.NSHB_ERR_WORKSPACE


def test_bad_destinations():
    s = fake((3, 5), (2, 5))
    assert clip(s, fake((3, 5), (2, 6), base=0x20000000)) == nshb.NSHB_ERR_SHAPE
    assert clip(s, fake((3, 5), (5, 2), base=0x20000000)) == nshb.NSHB_ERR_SHAPE
    assert clip(s, fake((3, 5), (2, 5), dtype=nshb.NSHB_F32)) == nshb.NSHB_ERR_PARAM     # in place, another type
    d = fake((3, 5), (2, 5))
    d[1].ld = 6
    assert clip(s, d) == nshb.NSHB_ERR_PARAM                                             # in place, another layout


def test_the_binding_refuses_what_the_library_cannot_see():
    with pytest.raises(ValueError, match="CUDA"):
        nshb.tensors([torch.zeros(3)])
    t = fake((3, 5))
    with pytest.raises(ValueError, match="CUDA"):
        nshb.grad_norm(t, torch.zeros(2), (WS, 1 << 20))
    with pytest.raises(ValueError, match="2 destinations for 1"):
        nshb.clip_grads(t, 1.0, TOTAL, (WS, 1 << 20), dst=fake((3, 5), (3, 5)))


# ------------------------------------------------------------------- 4-bit matrices


def fake4(*shapes, fmt=nshb.NSHB_NVFP4):
    arr = (nshb.nshb_fp4 * max(len(shapes), 1))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols, arr[i].format = r, c, fmt
        arr[i].codes, arr[i].scales, arr[i].global_ = 0x40000000 + 0x1000000 * i, 0x50000000 + 0x1000000 * i, 0x60000000
    arr._n = len(shapes)
    return arr


def quantize(x, q, transpose=0, ws=WS, ws_bytes=1 << 20, n=None):
    return nshb.lib().nshb_fp4_quantize(x, q, q._n if n is None else n, transpose, ws, ws_bytes, None)


def dequantize(q, x):
    return nshb.lib().nshb_fp4_dequantize(q, x, q._n, None)


def test_fp4_layout_and_sizes():
    assert ctypes.sizeof(nshb.nshb_fp4) == 48
    assert nshb.fp4_size(1, 1, nshb.NSHB_MXFP4) == (64, 512)
    assert nshb.fp4_size(129, 129, nshb.NSHB_MXFP4) == (129 * 128, 256 * 8)
    assert nshb.fp4_size(129, 129, nshb.NSHB_NVFP4) == (129 * 128, 256 * 16)
    assert nshb.fp4_size(0, 7, nshb.NSHB_MXFP4) == (0, 0)
    for args, code in (((-1, 1, 0), nshb.NSHB_ERR_SHAPE), ((1, -1, 0), nshb.NSHB_ERR_SHAPE), ((1, 1, 2), nshb.NSHB_ERR_DTYPE),
                       (((1 << 24) + 1, 1, 0), nshb.NSHB_ERR_UNSUPPORTED)):
        with pytest.raises(nshb.NshbError) as e:
            nshb.fp4_size(*args)
        assert e.value.status == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), nshb.NSHB_ERR_SHAPE),
    (dict(rows=3), nshb.NSHB_ERR_SHAPE),
    (dict(cols=6), nshb.NSHB_ERR_SHAPE),
    (dict(cols=(1 << 24) + 1), nshb.NSHB_ERR_UNSUPPORTED),
    (dict(format=2), nshb.NSHB_ERR_DTYPE),
    (dict(reserved=5), nshb.NSHB_ERR_PARAM),
    (dict(codes=None), nshb.NSHB_ERR_NULL),
    (dict(scales=None), nshb.NSHB_ERR_NULL),
    (dict(global_=None), nshb.NSHB_ERR_NULL),
    (dict(codes=0x40000008), nshb.NSHB_ERR_SHAPE),
    (dict(scales=0x50000004), nshb.NSHB_ERR_SHAPE),
    (dict(global_=0x60000002), nshb.NSHB_ERR_SHAPE),
])
def test_a_bad_4_bit_matrix_is_refused(change, code):
    x, q = fake((4, 5), (2, 5)), fake4((4, 5), (2, 5))
    for k, v in change.items():
        setattr(q[1], k, v)
    assert quantize(x, q) == dequantize(q, x) == code


def test_bad_quantize_arguments():
    x, q = fake((4, 5)), fake4((4, 5))
    assert quantize(x, q, transpose=1) == nshb.NSHB_ERR_SHAPE
    assert quantize(x, q, n=-1) == nshb.NSHB_ERR_SHAPE
    assert quantize(x, q, ws=None) == nshb.NSHB_ERR_NULL
    assert quantize(x, q, ws_bytes=64) == quantize(x, q, ws=WS + 64) == nshb.NSHB_ERR_WORKSPACE
    assert nshb.lib().nshb_fp4_quantize(x, None, 1, 0, WS, 1 << 20, None) == nshb.NSHB_ERR_NULL
    x[0].dtype = 3
    assert quantize(x, q) == dequantize(q, x) == nshb.NSHB_ERR_DTYPE
    with pytest.raises(ValueError, match="1 4-bit matrices for 2"):
        nshb.fp4_quantize(fake((4, 5), (4, 5)), q)


def matmul(a, b, d, ws=WS, ws_bytes=1 << 20, n=None):
    return nshb.lib().nshb_fp4_matmul(a, b, d, d._n if n is None else n, ws, ws_bytes, None)


def test_bad_products():
    a, b, d = fake4((4, 70)), fake4((6, 70)), fake((4, 6))
    assert matmul(a, b, fake((6, 4))) == matmul(a, None, d) == matmul(a, fake4((6, 69)), d) == nshb.NSHB_ERR_SHAPE
    assert matmul(a, fake4((6, 70), fmt=nshb.NSHB_MXFP4), d) == nshb.NSHB_ERR_DTYPE
    assert matmul(a, b, d, ws=None) == matmul(None, b, d) == matmul(a, b, None, n=1) == nshb.NSHB_ERR_NULL
    assert matmul(a, b, d, ws_bytes=128) == matmul(a, b, d, ws=WS + 16) == nshb.NSHB_ERR_WORKSPACE
    assert matmul(a, b, d, n=-1) == nshb.NSHB_ERR_SHAPE
    b[0].codes = None
    assert matmul(a, b, d) == nshb.NSHB_ERR_NULL
    with pytest.raises(ValueError, match="operands"):
        nshb.fp4_matmul(a, fake4((6, 70), (6, 70)), d, (WS, 1 << 20))


# --------------------------------------------------------- steps that take them


def fake_mats(*shapes):
    arr = (nshb.nshb_matrix * len(shapes))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols, arr[i].ld, arr[i].w_dtype, arr[i].z_index = r, c, c, nshb.NSHB_BF16, 0
        arr[i].W, arr[i].G, arr[i].M = 0x1000000, 0x2000000, 0x3000000
    arr._n = len(shapes)
    return arr


def test_scaled_step_refusals():
    m, p = fake_mats((64, 64)), nshb.params()
    call = lambda op, f, ws=0x9000000, nb=1 << 30: nshb.lib().nshb_step_scaled(op, m, 1, ctypes.byref(p), f, ws, nb, None)  # noqa: E731
    for op in (nshb.NSHB_OP_NEWTON_MUON, nshb.NSHB_OP_ADAMH, 99, -1):
        assert call(op, TOTAL) == nshb.NSHB_ERR_PARAM
    assert call(nshb.NSHB_OP_MUON, None) == call(nshb.NSHB_OP_MUON, TOTAL, ws=None) == nshb.NSHB_ERR_NULL
    assert call(nshb.NSHB_OP_MUON, TOTAL + 1) == nshb.NSHB_ERR_SHAPE
    assert call(nshb.NSHB_OP_MUON, TOTAL, nb=256) == nshb.NSHB_ERR_WORKSPACE


def test_newton_step_on_4_bit_inputs_refusals():
    m, p = fake_mats((100, 128)), nshb.params()
    call = lambda z, n=1, ws=0x9000000, nb=1 << 32: nshb.lib().newton_muon_step_fp4(m, 1, z, n, ctypes.byref(p), ws, nb, None)  # noqa: E731
    good = fake4((128, 77))
    assert call(None) == call(good, n=0) == call(good, ws=None) == nshb.NSHB_ERR_NULL
    assert call(good, nb=4096) == nshb.NSHB_ERR_WORKSPACE
    assert call(good, n=300) == nshb.NSHB_ERR_UNSUPPORTED
    assert call(fake4((128, 0))) == call(fake4((100, 77))) == call(fake4((192, 77))) == nshb.NSHB_ERR_SHAPE
    bad = fake4((128, 77))
    bad[0].scales = None
    assert call(bad) == nshb.NSHB_ERR_NULL
    m[0].z_index = 1
    assert call(good) == nshb.NSHB_ERR_PARAM


def test_an_array_of_another_kind_is_refused():
    t = fake((128, 64))
    ws = (WS, 1 << 20)
    q = (nshb.nshb_fp4 * 1)()
    m = (nshb.nshb_matrix * 1)()
    calls = [lambda: nshb.grad_norm(m, TOTAL, ws), lambda: nshb.grad_norm([t], TOTAL, ws),
             lambda: nshb.clip_grads(q, 1.0, TOTAL, ws), lambda: nshb.clip_grads(t, 1.0, TOTAL, ws, dst=m),
             lambda: nshb.scale_grads(m, TOTAL), lambda: nshb.fp4_quantize(t, t, ws),
             lambda: nshb.fp4_dequantize(t, t), lambda: nshb.fp4_matmul(t, q, t, ws),
             lambda: nshb.fp4_matmul(q, t, t, ws), lambda: nshb.fp4_matmul(q, None, q, ws),
             lambda: nshb.tensor_workspace(q),
             lambda: nshb.newton_muon_step_fp4(m, t, nshb.nshb_params(), ws)]
    for i, call in enumerate(calls):
        with pytest.raises(TypeError, match="an array of nshb_"):
            call()
            pytest.fail(f"call {i} went through")
