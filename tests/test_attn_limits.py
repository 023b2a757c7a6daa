"""The cache and attention calls at the edges of what they accept (CPU only: the checks come before any
HIP call; a call that passes them ends at the device check)."""
import ctypes

import pytest

import flatquant_transform_quant_amd as fq
from test_attn_api import B, D, DUMMY, H, HQ, INVAL, OK, RUNTIME, T, decode, decode_args, no_gpu, prefill, prefill_args, read, read_args, ref, tens, with_, write, write_args

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


@no_gpu
@pytest.mark.parametrize("d,most", [(64, 32 * (2 ** 24 - 1)), (72, 16 * (2 ** 24 - 1)), (128, 16 * (2 ** 24 - 1)), (256, 8 * (2 ** 24 - 1))])
def test_rows_that_a_cache_launch_can_hold(d, most):
    """A launch has fewer than 2^32 threads: 2^24 - 1 workgroups, of 32, 16 or 8 tokens each."""
    for n, want in ((most, RUNTIME), (most + 1, INVAL)):
        rows = tens(BF16, (n, 1, d))
        assert write(with_(write_args(h=1, d=d), k=rows, v=rows, slots=tens(fq.DT_INT32, (n,)))) == want
        assert read(with_(read_args(h=1, d=d), k=rows, v=rows)) == want


@no_gpu
@pytest.mark.parametrize("width", [2, 40])  # a workgroup a segment; a workgroup of the join a segment
def test_segments_that_a_decode_launch_can_hold(width):
    size = ctypes.c_uint64()
    for b, hq, h, want in ((65536, 255, 255, True), (65536, 256, 256, False), (16383, 1024, 1024, True), (16384, 1024, 1024, False),
                           (8191, 32768, 1024, True), (8192, 32768, 1024, False), (65536, 2000, 2, True)):
        rows = tens(BF16, (b, hq, 8))
        a = with_(decode_args(width=width, h=h, d=8), q=rows, out=rows, bt=tens(fq.DT_INT32, (b, width)), lens=tens(fq.DT_INT32, (b,)), ws=DUMMY,
                  size=2 ** 40)
        query = fq.lib.fq_attn_decode_get_workspace_size(ref(a["q"]), ref(a["kc"]), ref(a["bt"]), ctypes.byref(size))
        assert query == (OK if want else INVAL), (b, hq, h)
        assert decode(a) == (RUNTIME if want else INVAL), (b, hq, h)


@no_gpu
def test_workgroups_that_a_prompt_launch_can_hold():
    size = ctypes.c_uint64()
    for tq, b, hq, want in ((100, 65536, 255, True), (100, 65536, 256, False), (128 * 16383 - 129, 1, 1024, True), (128 * 16383, 1, 1024, False),
                            (127, 2 ** 14 - 1, 1024, True), (128, 2 ** 14 - 1, 1024, False)):
        a = prefill_args(tq=tq, tk=100, hq=hq, h=1, d=8, b=b)
        query = fq.lib.fq_attn_prefill_get_workspace_size(ref(a["q"]), ref(a["k"]), ref(a["cq"]), 1, ctypes.byref(size))
        assert query == (OK if want else INVAL), (tq, b, hq)
        assert prefill(a) == (RUNTIME if want else INVAL), (tq, b, hq)


@no_gpu
def test_scales_at_the_ends_of_the_range():
    for scale, want in ((2.0 ** 127, RUNTIME), (-2.0 ** 127, RUNTIME), (1e-300, RUNTIME), (-5e-324, RUNTIME), (1.001 * 2.0 ** 127, INVAL),
                        (-3e38, INVAL)):
        assert decode(with_(decode_args(), scale=scale)) == want
        assert prefill(with_(prefill_args(), scale=scale)) == want
