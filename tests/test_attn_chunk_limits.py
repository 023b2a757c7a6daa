"""Limits of attention of new tokens in the C ABI that its kernels need (CPU only)."""
import pytest

import flatquant_transform_quant_amd as fq
from test_attn_api import CODE, D, INVAL, RUNTIME, T, no_gpu, tens
from test_attn_chunk_api import HQ, args, call, with_


@no_gpu
@pytest.mark.parametrize("mode", list(CODE))
def test_scales(mode):
    """Integer codes enter the products 2^-9 of what they are; with f16 rows, which go in as they are, the scores' factor of 2^9 log2(e) times the
    scale is finite up to 2^118.  bf16 rows are brought to 2^14 at the most by a factor of their own, and the other formats need none."""
    for row in ("f16", "bf16"):
        if mode in ("f16", "bf16") and mode != row:
            continue
        x = tens(fq.DT_FLOAT16 if row == "f16" else fq.DT_BFLOAT16, (T, HQ, D))
        held = row == "f16" and mode in ("int8", "int4")
        for scale, ok in ((2.0 ** 118, True), (-2.0 ** 118, True), (2.0 ** 119, not held), (-2.0 ** 127, not held)):
            assert call(with_(args(mode), q=x, out=x, scale=scale)) == (RUNTIME if ok else INVAL), (row, scale)
