"""Refusals of the 8-bit entry points: every one on the host, before anything is enqueued (no GPU)."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_22_b200 as q
from bit_nf4_quantized_22_b200 import _lib
from bit_nf4_quantized_22_b200._lib import QLORA_EINVAL, QLORA_EUNSUPPORTED, QLORA_EWORKSPACE, QLORA_OK

P = ctypes.c_void_p(1 << 20)    # never dereferenced: the call is refused or empty


def odd(n):
    return ctypes.c_void_p((1 << 20) + n)


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_22_b200 import build
    build.build()
    return q.load()


def rows(rows=4, cols=100, ld=112, codes=1 << 20, scales=1 << 20):
    return ctypes.byref(_lib.Int8RowsC(rows, cols, ld, codes, scales))


BAD_ROWS = [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=1 << 31, ld=1 << 32), dict(ld=96), dict(ld=100),
            dict(codes=None), dict(codes=(1 << 20) + 8), dict(scales=None), dict(scales=(1 << 20) + 2)]


def weight(n=64, k=128):
    return ctypes.byref(_lib.NF4WeightC(n, k, 64, 1, 256, 0, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20))


def codebook():
    return (ctypes.c_float * 16)(*q.nf4_codebook().tolist())


def test_struct_layout():
    assert ctypes.sizeof(_lib.Int8RowsC) == 40 and _lib.Int8RowsC.codes.offset == 24


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_bad_rows(lib, bad):
    r = rows(**bad)
    big = 1 << 32
    assert lib.int8_quantize(P, 0, big, r, None, None) == QLORA_EINVAL
    assert lib.int8_dequantize(r, 0, P, None) == QLORA_EINVAL
    assert lib.int8_matmul(P, 0, big, r, rows(), None, P, 0, None, None) == QLORA_EINVAL
    assert lib.int8_matmul(P, 0, big, rows(), r, None, P, 0, None, None) == QLORA_EINVAL
    assert lib.int8_matmul_backward(P, 0, 4, r, P, P, 1 << 40, None, None) == QLORA_EINVAL
    assert lib.int8_matmul_backward_workspace_size(4, r) == 0
    assert lib.qlora_backward_int8(r, P, 4, weight(), codebook(), P, P, 8, 16.0, 1, None, P, P, P, P, 1 << 40,
                                   None, None) == QLORA_EINVAL


def test_quantize_refusals(lib):
    for dt in (-1, 3):
        assert lib.int8_quantize(P, dt, 100, rows(), None, None) == QLORA_EINVAL
        assert lib.int8_dequantize(rows(), dt, P, None) == QLORA_EINVAL
    assert lib.int8_quantize(P, 0, 99, rows(), None, None) == QLORA_EINVAL
    assert lib.int8_quantize(None, 0, 100, rows(), None, None) == QLORA_EINVAL
    assert lib.int8_quantize(odd(1), 0, 100, rows(), None, None) == QLORA_EINVAL
    assert lib.int8_quantize(odd(2), 2, 100, rows(), None, None) == QLORA_EINVAL
    assert lib.int8_dequantize(rows(), 0, None, None) == QLORA_EINVAL
    assert lib.int8_dequantize(rows(), 2, odd(2), None) == QLORA_EINVAL
    assert lib.int8_quantize(None, 0, 100, rows(rows=0), None, None) == QLORA_OK
    assert lib.int8_dequantize(rows(rows=0), 0, None, None) == QLORA_OK


def test_matmul_refusals(lib):
    def mm(x=P, xdt=0, ldx=100, x8=rows(), w=rows(rows=7), bias=None, y=P, ydt=0):
        return lib.int8_matmul(x, xdt, ldx, x8, w, bias, y, ydt, None, None)

    assert mm(w=rows(cols=101)) == QLORA_EINVAL
    assert mm(xdt=3) == QLORA_EINVAL and mm(ydt=-1) == QLORA_EINVAL
    assert mm(ldx=99) == QLORA_EINVAL and mm(x=odd(1)) == QLORA_EINVAL
    assert mm(y=None) == QLORA_EINVAL and mm(y=odd(1)) == QLORA_EINVAL and mm(y=odd(2), ydt=2) == QLORA_EINVAL
    assert mm(bias=odd(1)) == QLORA_EINVAL
    big = dict(cols=131073, ld=131088)
    assert mm(ldx=131073, x8=rows(**big), w=rows(**big)) == QLORA_EUNSUPPORTED
    assert mm(x8=rows(rows=0)) == QLORA_OK and mm(w=rows(rows=0)) == QLORA_OK


def test_input_gradient_refusals(lib):
    w = rows(rows=64)
    need = lib.int8_matmul_backward_workspace_size(5, w)
    assert need >= 2 * 5 * 64 + 20

    def bw(dy=P, dt=0, M=5, w=w, dx=P, ws=P, n=need):
        return lib.int8_matmul_backward(dy, dt, M, w, dx, ws, n, None, None)

    assert bw(dt=2) == QLORA_EINVAL and bw(M=-1) == QLORA_EINVAL and bw(w=rows(rows=0)) == QLORA_EINVAL
    assert bw(dy=None) == QLORA_EINVAL and bw(dx=None) == QLORA_EINVAL
    assert bw(dy=odd(1)) == QLORA_EINVAL and bw(dx=odd(1)) == QLORA_EINVAL
    assert bw(n=need - 1) == QLORA_EWORKSPACE and bw(ws=None) == QLORA_EWORKSPACE
    assert bw(w=rows(rows=131073)) == QLORA_EUNSUPPORTED
    assert lib.int8_matmul_backward_workspace_size(5, rows(rows=131073)) == 0
    assert bw(M=0, dy=None, dx=None, ws=None, n=0) == QLORA_OK


def test_checkpoint_refusals(lib):
    cb = codebook()
    x8 = rows(rows=4, cols=128, ld=128)
    need = lib.qlora_backward_int8_workspace_size(4, weight(), 8, 1)
    assert need > 0 and lib.qlora_backward_int8_workspace_size(4, weight(k=100), 8, 1) == 0

    def bw(x=x8, dy=P, M=4, w=weight(), r=8, alpha=16.0, g=1, ws=P, n=need):
        return lib.qlora_backward_int8(x, dy, M, w, cb, P, P, r, alpha, g, None, P, P, P, ws, n, None, None)

    assert bw(x=None) == QLORA_EINVAL
    assert bw(x=rows(rows=3, cols=128, ld=128)) == QLORA_EINVAL
    assert bw(x=rows(rows=4, cols=64, ld=64)) == QLORA_EINVAL
    assert bw(dy=None) == QLORA_EINVAL and bw(r=0) == QLORA_EINVAL and bw(g=2) == QLORA_EINVAL
    assert bw(alpha=float("nan")) == QLORA_EINVAL and bw(w=weight(n=60)) == QLORA_EUNSUPPORTED
    assert bw(n=need - 1) == QLORA_EWORKSPACE and bw(ws=None) == QLORA_EWORKSPACE
    assert bw(x=rows(rows=131073, cols=128, ld=128), M=131073, n=1 << 50) == QLORA_EUNSUPPORTED
    assert bw(x=rows(rows=0, cols=128, ld=128), M=0) == QLORA_OK


def test_binding_refusals(lib):
    x = torch.zeros(4, 64)
    r8 = q.Int8Rows(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError):
        q.int8_quantize(x)
    with pytest.raises(TypeError):
        q.int8_matmul(x, r8)
    with pytest.raises(TypeError):
        q.int8_matmul(r8, r8)
    with pytest.raises(TypeError):
        q.int8_matmul_backward(x, r8)
    with pytest.raises(TypeError):
        q.int8_dequantize(r8)
    with pytest.raises(TypeError):
        r8.c_struct()


def test_unaligned_workspaces(lib):
    for n in (1, 4, 8):
        assert lib.int8_matmul_backward(P, 0, 4, rows(), P, odd(n), 1 << 40, None, None) == QLORA_EINVAL
        assert lib.qlora_backward_int8(rows(4, 128, 128), P, 4, weight(), codebook(), P, P, 8, 16.0, 1, None, P, P, P,
                                       odd(n), 1 << 40, None, None) == QLORA_EINVAL
