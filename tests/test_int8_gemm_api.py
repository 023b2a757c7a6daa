"""The int8 consumer GEMM of the C ABI: what it refuses (CPU only: the checks come before any HIP call; a call that passes
them ends at the device check)."""
import ctypes

import pytest
import torch

import flatquant_transform_quant_amd as fq
from test_attn_api import DUMMY, INVAL, NULLP, OK, RUNTIME, no_gpu, tens


def args(T=32, O=16, H=256, cdt=fq.DT_BFLOAT16):
    return [tens(fq.DT_INT8, (T, H)), tens(fq.DT_FLOAT32, (T,)), tens(fq.DT_INT8, (O, H)), tens(fq.DT_FLOAT32, (O,)), tens(cdt, (T, O))]


def call(a):
    return fq.lib.fq_int8_gemm(*(None if t is None else ctypes.addressof(t) for t in a), None)


def but(i, t, **kw):
    a = args(**kw)
    a[i] = t
    return a


def test_missing():
    for i, t in enumerate(args()):
        assert call(but(i, None)) == NULLP
        assert call(but(i, tens(t.dtype, list(t.shape)[:t.ndim], data=0))) == NULLP


def test_refused():
    I8, F32, B16 = fq.DT_INT8, fq.DT_FLOAT32, fq.DT_BFLOAT16
    for a in (but(0, tens(fq.DT_INT4, (32, 256))), but(2, tens(fq.DT_FLOAT8_E4M3FN, (16, 256))), but(2, tens(I8, (16, 272))), but(0, tens(I8, (32, 256), (512, 1))),
              but(2, tens(I8, (16, 256), (1, 16))), but(0, tens(I8, (32 * 256,))), but(1, tens(F32, (31,))), but(1, tens(F32, (32, 1))), but(1, tens(B16, (32,))),
              but(3, tens(F32, (32,))), but(1, tens(F32, (32,), (2,))), but(4, tens(I8, (32, 16))), but(4, tens(B16, (16, 32))), but(4, tens(B16, (32, 16), (32, 1))),
              but(0, tens(I8, (32, 256), data=DUMMY + 8)), but(2, tens(I8, (16, 256), data=DUMMY + 1)), but(1, tens(F32, (32,), data=DUMMY + 2)),
              but(4, tens(B16, (32, 16), data=DUMMY + 1)), but(4, tens(F32, (32, 16), data=DUMMY + 2))):
        assert call(a) == INVAL
    for H in (0, 8, 24, 100, 2 ** 17):
        assert call(args(H=H)) == INVAL, H
    for T, O in ((2 ** 26, 1), (1, 2 ** 26), (2 ** 18, 2 ** 19)):
        assert call(args(T=T, O=O)) == INVAL


@no_gpu
def test_accepted():
    for cdt in (fq.DT_BFLOAT16, fq.DT_FLOAT16, fq.DT_FLOAT32):
        assert call(args(cdt=cdt)) == RUNTIME
    for T, O, H in ((1, 1, 16), (2 ** 26 - 1, 1, 2 ** 17 - 16), (1, 2 ** 26 - 1, 48), (2 ** 18 - 128, 2 ** 19, 16)):
        assert call(args(T, O, H)) == RUNTIME
    assert call(but(4, tens(fq.DT_BFLOAT16, (32, 16), data=DUMMY + 2))) == RUNTIME


def test_nothing_to_do():
    z = lambda t, *s: tens(t, s, data=0)  # noqa: E731
    assert call([z(fq.DT_INT8, 0, 256), z(fq.DT_FLOAT32, 0), *args()[2:4], z(fq.DT_BFLOAT16, 0, 16)]) == OK
    assert call([*args()[:2], z(fq.DT_INT8, 0, 256), z(fq.DT_FLOAT32, 0), z(fq.DT_BFLOAT16, 32, 0)]) == OK


def test_binding_refuses():
    a, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="runs on a GPU"):
        fq.int8_gemm(a, s, a, s)
