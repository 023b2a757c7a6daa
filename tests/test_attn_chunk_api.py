"""Attention of new tokens in the C ABI: what it refuses, and the workspace it asks for (CPU only)."""
import ctypes

import pytest
import torch

import flatquant_transform_quant_amd as fq
from test_attn_api import CODE, D, DUMMY, H, INVAL, NULLP, OK, P, PAGES, RUNTIME, T, cache, no_gpu, ref, tens

B, HQ = 3, 4
BF16, F32, I32 = fq.DT_BFLOAT16, fq.DT_FLOAT32, fq.DT_INT32


def args(mode="int8", t=T, hq=HQ, b=B, width=2, window=0, sinks=0, **kw):
    d = kw.get("d", D)
    return dict(cache(mode, **kw), q=tens(BF16, (t, hq, d)), bt=tens(I32, (b, width)), cu=tens(I32, (b + 1,)), lens=tens(I32, (b,)), window=window, sinks=sinks,
                scale=0.0, out=tens(BF16, (t, hq, d)), lse=None, ws=None, size=0)


def need(a):
    size = ctypes.c_uint64(1 << 60)
    p = lambda n: None if a[n] is None else ctypes.addressof(a[n])  # noqa: E731
    st = fq.lib.fq_attn_chunk_get_workspace_size(p("q"), p("kc"), p("bt"), p("cu"), a["window"], a["sinks"], ctypes.byref(size))
    return st, size.value


def call(a):
    p = lambda n: None if a[n] is None else ctypes.addressof(a[n])  # noqa: E731
    return fq.lib.fq_attn_chunk(*(p(n) for n in ("q", "kc", "ks", "vc", "vs", "bt", "cu", "lens")), a["window"], a["sinks"], a["scale"], p("out"), p("lse"),
                                a["ws"], a["size"], None)


def with_(a, **kw):
    return dict(a, **kw)


def test_missing():
    for n in ("q", "kc", "vc", "ks", "vs", "bt", "cu", "lens", "out"):
        assert call(with_(args(), **{n: None})) == NULLP, n
        t = args()[n]
        assert call(with_(args(), **{n: fq.make_tensor(0, t.dtype, list(t.shape)[:t.ndim])})) == NULLP, n
    assert call(with_(args(), lse=fq.make_tensor(0, F32, (T, HQ)))) == NULLP
    for n in ("q", "kc", "bt", "cu"):
        assert need(with_(args(), **{n: None}))[0] == NULLP


def test_refused():
    a = args()
    bad = dict(
        q=[tens(F32, (T, HQ, D)), tens(fq.DT_FLOAT16, (T, HQ, D)), tens(BF16, (T, 3, D)), tens(BF16, (T, HQ, D + 8)), tens(BF16, (T, HQ)), tens(BF16, (T, HQ, D), (HQ * D + 4, D, 1)),
           tens(BF16, (T, HQ, D), data=DUMMY + 8)],
        out=[tens(fq.DT_FLOAT16, (T, HQ, D)), tens(BF16, (T + 1, HQ, D)), tens(BF16, (T, HQ, D), (0, D, 1)), tens(BF16, (T, HQ, D), (HQ * D, 8, 1))],
        bt=[tens(F32, (B, 2)), tens(I32, (B + 1, 2)), tens(I32, (B, 2), (4, 2)), tens(I32, (B,))],
        cu=[tens(F32, (B + 1,)), tens(I32, (B,)), tens(I32, (1,)), tens(I32, (B + 1,), (2,)), tens(I32, (B + 1, 1))],
        lens=[tens(I32, (B + 1,)), tens(F32, (B,)), tens(I32, (B,), (2,))],
        lse=[tens(F32, (T, HQ + 1)), tens(BF16, (T, HQ)), tens(F32, (T, HQ), (HQ + 1, 1))],
        window=[-1, -2 ** 31], sinks=[-1], scale=[1e39, float("nan"), float("inf")],
        kc=[tens(fq.DT_INT8, (PAGES, H, 24, D)), tens(fq.DT_INT8, (PAGES, H, P, D + 8))],
    )
    for n, ts in bad.items():
        for i, t in enumerate(ts):
            assert call(with_(a, **{n: t})) == INVAL, (n, i)
    assert call(args("f16")) == INVAL  # bf16 queries over an f16 cache
    assert need(with_(a, window=-1))[0] == INVAL and need(with_(a, sinks=-1))[0] == INVAL


@no_gpu
def test_accepted():
    for mode in CODE:
        if mode != "f16":
            assert call(args(mode)) == RUNTIME
    assert call(args(window=5, sinks=3)) == RUNTIME
    assert call(args(window=2 ** 31 - 1, sinks=2 ** 31 - 1)) == RUNTIME
    assert call(with_(args(), lse=tens(F32, (T, HQ)))) == RUNTIME
    assert call(with_(args(), bt=fq.make_tensor(0, I32, (B, 0)))) == RUNTIME


def test_no_rows():
    z = fq.make_tensor(0, BF16, (0, HQ, D))
    assert call(with_(args(), q=z, out=z)) == OK


def test_the_workspace():
    """None where every row tile is one workgroup's; two parts a run otherwise, of a row tile with two more values a row."""
    assert need(args()) == (OK, 0)
    st, big = need(args(t=64, width=4096))
    assert st == OK and big == 2 * 512 * 64 * (D + 2) * 4  # (22 tokens of 2 heads a sequence: row tiles of 64)
    a = args(t=64, width=4096)
    assert call(a) == NULLP
    assert call(with_(a, ws=DUMMY, size=big - 1)) == INVAL and call(with_(a, ws=DUMMY + 4, size=big)) == INVAL
    # a window bounds the walks, whatever the table's reach
    few = need(args(t=3, b=1, width=4096, window=100, sinks=4))
    assert few == (OK, 0)
    assert need(args(t=3, b=1, width=4096))[1] > 0
    # heads above 128 run one workgroup a CU
    assert need(args(t=64, width=4096, d=256))[1] == 2 * 256 * 64 * 258 * 4


@no_gpu
def test_sizes_that_are_counted_in_31_bits():
    size = (1 << 64) - 1
    for t, b, width, ok in ((2 ** 20, 1, 2 ** 15, True), (2 ** 21, 1, 2 ** 20, False), (2 ** 31 - 65537, 1, 1, True), (2 ** 31 - 65536, 1, 1, False),
                            (1, 65536, 2 ** 22, True), (65536, 65536, 2 ** 22, False), (1, 1, 2 ** 27 - 4096, False), (1, 1, 2 ** 27 - 4097, True)):
        a = with_(args(t=t, b=b, width=width, hq=16, h=1, pages=7), ws=DUMMY, size=size)
        assert call(a) == (RUNTIME if ok else INVAL), (t, b, width)
        assert need(a)[0] == (OK if ok else INVAL)


def test_binding_refuses():
    c = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    q, i = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="runs on a GPU"):
        fq.attn_chunk(q, c, i[None], i, i[:1])
