"""The norm and rotation calls of the C ABI: what they refuse (CPU only: the checks come before any HIP call; a call
that passes them ends at the device check)."""
import pytest
import torch

import flatquant_transform_quant_amd as fq
from test_attn_api import D, DUMMY, H, INVAL, NULLP, OK, RUNTIME, T, cache, no_gpu, ref, tens

HQ = 4
BF16, F16, F32, I32 = fq.DT_BFLOAT16, fq.DT_FLOAT16, fq.DT_FLOAT32, fq.DT_INT32


def rope_args(dt=BF16, t=T, d=D, r=D):
    rows = lambda h: tens(dt, (t, h, d))  # noqa: E731
    return dict(q=rows(HQ), k=rows(H), wq=None, wk=None, eps=1e-6, pos=tens(I32, (t,)), f=tens(F32, (r // 2,)), axes=None, turn=0, qo=rows(HQ), ko=rows(H))


def rope(a):
    return fq.lib.fq_qk_rope(*(_p(a[n]) for n in ("q", "k", "wq", "wk")), a["eps"], *(_p(a[n]) for n in ("pos", "f", "axes")), a["turn"], _p(a["qo"]), _p(a["ko"]), None)


def append_args(mode="int8", **kw):
    c = cache(mode, **kw)
    return dict(rope_args(), v=tens(BF16, (T, H, D)), slots=tens(I32, (T,)), clip=1.0, dmax=0.0, **c)


def append(a):
    return fq.lib.fq_kv_append(*(_p(a[n]) for n in ("q", "k", "v", "slots", "wq", "wk")), a["eps"], *(_p(a[n]) for n in ("pos", "f", "axes")), a["turn"],
                               a["clip"], a["dmax"], *(_p(a[n]) for n in ("kc", "ks", "vc", "vs", "qo")), None)


def _p(t):
    import ctypes
    return None if t is None else ctypes.addressof(t)


def with_(a, **kw):
    return dict(a, **kw)


BOTH = [(rope_args, rope), (append_args, append)]


@pytest.mark.parametrize("make,call", BOTH)
def test_missing(make, call):
    for n in ("q", "qo", "pos", "f"):
        t = make()[n]
        empty = fq.make_tensor(0, t.dtype, list(t.shape)[:t.ndim])
        assert call(with_(make(), **{n: empty})) == NULLP, n
    for n in ("qo", "pos", "f"):
        assert call(with_(make(), **{n: None})) == NULLP, n
    for n, shape in (("wq", (D,)), ("wk", (D,)), ("axes", (D // 2,))):
        assert call(with_(make(), **{n: fq.make_tensor(0, I32 if n == "axes" else F32, shape)})) == NULLP
    assert rope(with_(rope_args(), q=None, k=None)) == NULLP
    assert rope(with_(rope_args(), ko=None)) == NULLP
    for n in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert append(with_(append_args(), **{n: None})) == NULLP, n


@pytest.mark.parametrize("make,call", BOTH)
def test_refused(make, call):
    a = make()
    bad = dict(
        q=[tens(F32, (T, HQ, D)), tens(F16, (T, HQ, D)), tens(BF16, (T + 1, HQ, D)), tens(BF16, (T, HQ, D + 8)), tens(BF16, (T, HQ, D), (HQ * D + 4, D, 1)),
           tens(BF16, (T, HQ, D), (HQ * D, D, 2)), tens(BF16, (T, HQ, D), data=DUMMY + 8), tens(BF16, (T, HQ * D)), tens(BF16, (T, 65537, D))],
        qo=[tens(F16, (T, HQ, D)), tens(BF16, (T, HQ + 1, D)), tens(BF16, (T, HQ, D), (0, D, 1)), tens(BF16, (T, HQ, D), (HQ * D, D - 8, 1))],
        k=[tens(F16, (T, H, D)), tens(BF16, (T, H)), tens(BF16, (T - 1, H, D))],
        wq=[tens(I32, (D,)), tens(F32, (D - 1,)), tens(F32, (1, D)), tens(F32, (D,), (2,)), tens(F32, (D,), data=DUMMY + 2), tens(BF16, (D,), data=DUMMY + 1)],
        wk=[tens(I32, (D,)), tens(F32, (D + 1,))],
        eps=[0.0, -1.0, 1e-60, 1e60, float("nan"), float("inf")],
        pos=[tens(F32, (T,)), tens(I32, (T + 1,)), tens(I32, (1, T)), tens(I32, (T,), (2,)), tens(I32, (T,), data=DUMMY + 2)],
        f=[tens(BF16, (D // 2,)), tens(F32, (D // 2 + 4,)), tens(F32, (D // 2 - 1,)), tens(F32, (2,)), tens(F32, (1, D // 2)), tens(F32, (D // 2,), (2,))],
        axes=[tens(I32, (D // 2,))],  # (with positions of one dimension)
    )
    for n, ts in bad.items():
        for i, t in enumerate(ts):
            assert call(with_(a, **{n: t})) == INVAL, (n, i)
    ax = tens(I32, (D // 2,))
    for p in (tens(I32, (0, T)), tens(I32, (17, T)), tens(I32, (3, T + 1)), tens(I32, (3, T), (T, 2)), tens(F32, (3, T)), tens(I32, (3, T), (2 ** 40, 1))):
        assert call(with_(a, pos=p, axes=ax)) == INVAL
    for x in (tens(F32, (D // 2,)), tens(I32, (D // 2 - 1,)), tens(I32, (D // 2,), (2,))):
        assert call(with_(a, pos=tens(I32, (3, T)), axes=x)) == INVAL


def test_refused_by_one():
    rows = lambda t, h, d: tens(BF16, (t, h, d))  # noqa: E731
    for d in (4, 12, 264):
        a = with_(rope_args(), q=rows(T, HQ, d), k=rows(T, H, d), qo=rows(T, HQ, d), ko=rows(T, H, d), f=tens(F32, (0,)))
        assert rope(a) == INVAL
    assert rope(with_(rope_args(), ko=tens(BF16, (T, H, D), (0, D, 1)))) == INVAL
    a = append_args()
    for n, ts in dict(v=[tens(F16, (T, H, D)), tens(BF16, (T, H + 1, D))], slots=[tens(F32, (T,)), tens(I32, (T + 1,))], clip=[0.0, 1.5, float("nan")],
                      dmax=[1.0, 13.0, float("nan")], k=[tens(BF16, (T, H + 1, D))]).items():
        for t in ts:
            assert append(with_(a, **{n: t})) == INVAL, n
    assert append(append_args("f16")) == INVAL  # bf16 rows into an f16 cache


@no_gpu
@pytest.mark.parametrize("make,call", BOTH)
def test_accepted(make, call):
    a = make()
    assert call(a) == RUNTIME
    assert call(with_(a, q=None, qo=None)) == RUNTIME
    assert call(with_(a, f=fq.make_tensor(0, F32, (0,)))) == RUNTIME
    assert call(with_(a, q=tens(BF16, (T, HQ, D), ((HQ + 4) * D, D, 1)), wq=tens(F16, (D,)), wk=tens(F32, (D,)), turn=1)) == RUNTIME
    assert call(with_(a, pos=tens(I32, (3, T), (T + 7, 1)), axes=tens(I32, (D // 2,)))) == RUNTIME
    assert call(with_(a, qo=a["q"])) == RUNTIME
    assert call(with_(a, q=tens(BF16, (T, 0, D), data=0), qo=tens(BF16, (T, 0, D), data=0))) == RUNTIME


def test_no_rows():
    z = lambda h: fq.make_tensor(0, BF16, (0, h, D))  # noqa: E731
    a = with_(rope_args(), q=z(HQ), k=z(H), qo=z(HQ), ko=z(H), pos=fq.make_tensor(0, I32, (0,)))
    assert rope(a) == OK
    assert append(with_(append_args(), q=z(HQ), k=z(H), v=z(H), qo=z(HQ), slots=fq.make_tensor(0, I32, (0,)), pos=fq.make_tensor(0, I32, (0,)))) == OK


@no_gpu
@pytest.mark.parametrize("d,most", [(64, 32 * (2 ** 24 - 1)), (128, 16 * (2 ** 24 - 1)), (256, 8 * (2 ** 24 - 1))])
def test_rows_that_a_launch_can_hold(d, most):
    for n, want in ((most, RUNTIME), (most + 1, INVAL)):
        rows = tens(BF16, (n, 1, d))
        assert rope(with_(rope_args(), q=rows, k=None, qo=rows, ko=None, pos=tens(I32, (n,)), f=tens(F32, (d // 2,)))) == want


def test_binding_refuses():
    cache_ = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    rows, pos, f = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="runs on a GPU"):
        fq.qk_rope(rows, rows, pos, f)
    with pytest.raises(ValueError, match="runs on a GPU"):
        fq.kv_append(cache_, rows, rows, rows, pos, pos, f)
    with pytest.raises(ValueError, match="neither"):
        fq.qk_rope(None, None, pos, f)
