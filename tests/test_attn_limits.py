"""The cache and attention calls at the edges of what they accept (CPU only: the checks come before any
HIP call; a call that passes them ends at the device check)."""
import ctypes

import pytest

import flatquant_transform_quant_amd as fq
from test_attn_api import B, D, H, HQ, INVAL, OK, RUNTIME, T, decode, decode_args, no_gpu, prefill, prefill_args, read, read_args, ref, tens, with_, write, write_args

BF16 = fq.DT_BFLOAT16
# name, key, rows, heads, call
OUTPUTS = [("read", "k", T, H), ("read", "v", T, H), ("decode", "out", B, HQ), ("prefill", "out", T, HQ)]
CALLS = {"read": (read_args, read), "decode": (decode_args, decode), "prefill": (prefill_args, prefill)}


@pytest.mark.parametrize("name,key,n,h", OUTPUTS)
def test_output_elements_over_each_other_are_refused(name, key, n, h):
    make, call = CALLS[name]
    for strides in ((0, D, 1), (h * D, 0, 1), (0, 0, 1), (h * D - 8, D, 1), (h * D, D - 8, 1), (D, D, 1), (D - 8, n * D, 1), (D, n * D - 8, 1),
                    (8, 2 ** 39, 1), (2 ** 39, 8, 1)):
        assert call(with_(make(), **{key: tens(BF16, (n, h, D), strides)})) == INVAL, strides


@no_gpu
@pytest.mark.parametrize("name,key,n,h", OUTPUTS)
def test_output_elements_apart_are_accepted(name, key, n, h):
    make, call = CALLS[name]
    for strides in ((h * D, D, 1), ((h + 1) * D, D, 1), (h * (D + 8), D + 8, 1), (D, n * D, 1), (D + 8, n * (D + 8), 1), (D, 2 ** 39, 1), (2 ** 39, D, 1)):
        assert call(with_(make(), **{key: tens(BF16, (n, h, D), strides)})) == RUNTIME, strides
    # inputs may repeat rows
    if name != "read":
        assert call(with_(make(), q=tens(BF16, (n, h, D), (0, D, 1)))) == RUNTIME
        assert call(with_(make(), q=tens(BF16, (n, h, D), (0, 0, 1)))) == RUNTIME


@no_gpu
def test_the_stride_of_a_single_row_or_head_does_not_count():
    for strides in ((0, D, 1), (8, D, 1)):
        assert decode(with_(decode_args(), q=tens(BF16, (1, HQ, D)), out=tens(BF16, (1, HQ, D), strides), bt=tens(fq.DT_INT32, (1, 2)),
                            lens=tens(fq.DT_INT32, (1,)))) == RUNTIME
        a = prefill_args(hq=1, h=1)
        assert prefill(with_(a, out=tens(BF16, (T, 1, D), (D, 0, 1)))) == RUNTIME
        assert prefill(with_(a, out=tens(BF16, (T, 1, D), (D - 8, 0, 1)))) == INVAL
