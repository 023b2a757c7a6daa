"""The cache and attention calls of the C ABI: what they refuse, in which order, and the workspace they
ask for (CPU only: the checks come before any HIP call; a call that passes them ends at the
device check)."""
import ctypes

import pytest
import torch

import flatquant_transform_quant_amd as fq

DUMMY = 0x10000  # never dereferenced by the checks
NULLP, INVAL, OK, RUNTIME = fq.FQ_ERR_PARAM_NULLPTR, fq.FQ_ERR_PARAM_INVALID, fq.FQ_SUCCESS, fq.FQ_ERR_RUNTIME
PAGES, H, P, D, T, B, HQ = 5, 2, 16, 64, 7, 3, 4

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="a call with made-up pointers must not reach a device")


def tens(dtype, shape, strides=None, data=DUMMY):
    return fq.make_tensor(data, dtype, shape, strides)


def ref(t):
    return ctypes.byref(t) if t is not None else None


CODE = {"f16": fq.DT_FLOAT16, "bf16": fq.DT_BFLOAT16, "int8": fq.DT_INT8, "e4m3": fq.DT_FLOAT8_E4M3FN, "int4": fq.DT_INT4,
        "fp4": fq.DT_FLOAT4_E2M1}


def cache(mode="int8", pages=PAGES, h=H, p=P, d=D, data=DUMMY):
    """The four cache tensors of a call."""
    c = lambda: tens(CODE[mode], (pages, h, p, d), data=data)  # noqa: E731
    if mode in ("f16", "bf16"):
        s = lambda: None  # noqa: E731
    elif mode == "fp4":
        s = lambda: tens(fq.DT_FLOAT8_E8M0, (pages, h, p, 2 * (-(-d // 64))))  # noqa: E731
    else:
        s = lambda: tens(fq.DT_FLOAT32, (pages, h, p))  # noqa: E731
    return {"kc": c(), "ks": s(), "vc": c(), "vs": s()}


def write_args(mode="int8", **kw):
    return dict(cache(mode, **kw), k=tens(fq.DT_BFLOAT16, (T, H, D)), v=tens(fq.DT_BFLOAT16, (T, H, D)), slots=tens(fq.DT_INT32, (T,)),
                clip=1.0, dmax=0.0)


def write(a):
    return fq.lib.fq_kv_write(ref(a["k"]), ref(a["v"]), ref(a["slots"]), a["clip"], a["dmax"], ref(a["kc"]), ref(a["ks"]), ref(a["vc"]),
                              ref(a["vs"]), None)


def read_args(mode="int8", **kw):
    return dict(cache(mode, **kw), bt=tens(fq.DT_INT32, (B, 2)), cu=tens(fq.DT_INT32, (B + 1,)), k=tens(fq.DT_BFLOAT16, (T, H, D)),
                v=tens(fq.DT_BFLOAT16, (T, H, D)))


def read(a):
    return fq.lib.fq_kv_read(ref(a["kc"]), ref(a["ks"]), ref(a["vc"]), ref(a["vs"]), ref(a["bt"]), ref(a["cu"]), ref(a["k"]), ref(a["v"]), None)


def decode_args(mode="int8", width=2, **kw):
    return dict(cache(mode, **kw), q=tens(fq.DT_BFLOAT16, (B, HQ, D)), bt=tens(fq.DT_INT32, (B, width)), lens=tens(fq.DT_INT32, (B,)),
                out=tens(fq.DT_BFLOAT16, (B, HQ, D)), lse=None, scale=0.0, ws=None, size=0)


def decode(a):
    return fq.lib.fq_attn_decode(ref(a["q"]), ref(a["kc"]), ref(a["ks"]), ref(a["vc"]), ref(a["vs"]), ref(a["bt"]), ref(a["lens"]), a["scale"],
                                 ref(a["out"]), ref(a["lse"]), a["ws"], a["size"], None)


def prefill_args(tq=T, tk=T, hq=HQ, h=H, d=D, dt=fq.DT_BFLOAT16, b=B):
    return dict(q=tens(dt, (tq, hq, d)), k=tens(dt, (tk, h, d)), v=tens(dt, (tk, h, d)), cq=tens(fq.DT_INT32, (b + 1,)),
                ck=tens(fq.DT_INT32, (b + 1,)), causal=1, scale=0.0, out=tens(dt, (tq, hq, d)), lse=None, ws=None, size=0)


def prefill(a):
    return fq.lib.fq_attn_prefill(ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["cq"]), ref(a["ck"]), a["causal"], a["scale"], ref(a["out"]),
                                  ref(a["lse"]), a["ws"], a["size"], None)


CALLS = {"write": (write_args, write), "read": (read_args, read), "decode": (decode_args, decode), "prefill": (prefill_args, prefill)}


def with_(args, **kw):
    return dict(args, **kw)


@no_gpu
@pytest.mark.parametrize("mode", list(CODE))
def test_valid_calls_pass_the_checks(mode):
    rows = fq.DT_FLOAT16 if mode == "f16" else fq.DT_BFLOAT16
    fix = lambda a, n: {k: (tens(rows, (B if n == "decode" else T, HQ if n == "decode" else H, D)) if k in ("k", "v", "q", "out") else v)  # noqa: E731
                        for k, v in a.items()}
    for name in ("write", "read", "decode"):
        make, call = CALLS[name]
        assert call(fix(make(mode), name)) == RUNTIME, name
    assert "gfx950" in fq.fq_last_error()
    assert prefill(prefill_args()) == RUNTIME
    assert prefill(prefill_args(dt=fq.DT_FLOAT16, d=8)) == RUNTIME


@pytest.mark.parametrize("name,key", [(n, k) for n, ks in (("write", "k v slots kc ks vc vs"), ("read", "kc ks vc vs bt cu k v"),
                                                         ("decode", "q kc ks vc vs bt lens out"), ("prefill", "q k v cq ck out"))
                                      for k in ks.split()])
def test_missing_tensors(name, key):
    make, call = CALLS[name]
    assert call(with_(make(), **{key: None})) == NULLP
    t = make()[key]
    gone = fq.make_tensor(0, t.dtype, list(t.shape[:t.ndim]), list(t.strides[:t.ndim]))
    assert call(with_(make(), **{key: gone})) == NULLP
    if name in ("decode", "prefill"):
        assert call(with_(make(), lse=tens(fq.DT_FLOAT32, (B, HQ), data=0))) == NULLP


def test_empty_calls_do_nothing():
    none = lambda *s: tens(fq.DT_BFLOAT16, s, data=0)  # noqa: E731
    assert write(with_(write_args(), k=none(0, H, D), v=none(0, H, D), slots=tens(fq.DT_INT32, (0,), data=0))) == OK
    assert read(with_(read_args(), k=none(0, H, D), v=none(0, H, D))) == OK
    assert read(with_(read_args(), bt=tens(fq.DT_INT32, (0, 2), data=0), cu=tens(fq.DT_INT32, (1,)))) == OK
    assert decode(with_(decode_args(), q=none(0, HQ, D), out=none(0, HQ, D), bt=tens(fq.DT_INT32, (0, 2), data=0),
                        lens=tens(fq.DT_INT32, (0,), data=0))) == OK
    assert prefill(with_(prefill_args(), q=none(0, HQ, D), out=none(0, HQ, D))) == OK


@pytest.mark.parametrize("name", ["write", "read", "decode"])
def test_cache_shapes_refused(name):
    make, call = CALLS[name]
    for kw in (dict(p=8), dict(p=24), dict(p=2048), dict(d=12), dict(d=264), dict(d=4), dict(h=1025), dict(pages=2 ** 28)):
        assert call(make("int8", **kw)) == INVAL, kw
    assert call(make("fp4", d=48)) == INVAL  # whole groups of 32
    ok = make("int8")
    assert call(with_(ok, kc=tens(fq.DT_FLOAT8_E5M2, (PAGES, H, P, D)), vc=tens(fq.DT_FLOAT8_E5M2, (PAGES, H, P, D)))) == INVAL
    assert call(with_(ok, vc=tens(fq.DT_FLOAT8_E4M3FN, (PAGES, H, P, D)))) == INVAL  # the sides differ
    assert call(with_(ok, vc=tens(fq.DT_INT8, (PAGES + 1, H, P, D)))) == INVAL
    assert call(with_(ok, ks=tens(fq.DT_FLOAT16, (PAGES, H, P)))) == INVAL
    assert call(with_(ok, vs=tens(fq.DT_FLOAT32, (PAGES, H, P + 1)))) == INVAL
    assert call(with_(ok, ks=tens(fq.DT_FLOAT32, (PAGES, H, P), data=DUMMY + 4))) == INVAL
    assert call(with_(ok, kc=tens(fq.DT_INT8, (PAGES, H, P, D), data=DUMMY + 8))) == INVAL
    assert call(with_(ok, kc=tens(fq.DT_INT8, (PAGES, H, P, D), [H * P * D + 8, P * D, D, 1]))) == INVAL  # pages 16-byte aligned
    assert call(with_(ok, kc=tens(fq.DT_INT8, (PAGES, H, P, D), [H * P * D, D, H * D, 1]))) == INVAL  # inner dimensions contiguous
    assert call(with_(ok, kc=tens(fq.DT_INT8, (PAGES, H, P, D), [0, P * D, D, 1]))) == INVAL  # pages over each other
    assert call(with_(make("fp4"), ks=tens(fq.DT_FLOAT8_E8M0, (PAGES, H, P, 4)))) == INVAL


@pytest.mark.parametrize("name,keys", [("write", "k v"), ("read", "k v"), ("decode", "q out"), ("prefill", "q k v out")])
def test_rows_refused(name, keys):
    make, call = CALLS[name]
    for key in keys.split():
        t = make()[key]
        n, h, d = t.shape[:3]
        for bad in (tens(fq.DT_FLOAT32, (n, h, d)), tens(t.dtype, (n, h * d)), tens(t.dtype, (n, h + 1, d)), tens(t.dtype, (n, h, d - 8)),
                    tens(t.dtype, (n, h, d), [h * d + 4, d, 1]), tens(t.dtype, (n, h, d), [h * d, d + 4, 1]),
                    tens(t.dtype, (n, h, d), [2 * h * d, 2 * d, 2]), tens(t.dtype, (n, h, d), [-h * d, d, 1]),
                    tens(t.dtype, (n, h, d), data=DUMMY + 8), tens(fq.DT_FLOAT16, (n, h, d))):
            if name in ("write", "read") and key == "k" and bad.dtype == fq.DT_FLOAT16:
                continue  # (then v is the one that differs)
            assert call(with_(make(), **{key: bad})) == INVAL, (name, key, list(bad.shape), list(bad.strides), bad.dtype)


def test_scalars_refused():
    for clip in (0.0, -0.5, 1.5, float("nan")):
        assert write(with_(write_args(), clip=clip)) == INVAL
    for dmax in (5.9, 12.1, -6.0, float("nan")):
        assert write(with_(write_args("fp4"), dmax=dmax)) == INVAL
    for scale in (float("inf"), float("nan"), 1e300):
        assert decode(with_(decode_args(), scale=scale)) == INVAL
        assert prefill(with_(prefill_args(), scale=scale)) == INVAL


def test_index_tensors_refused():
    assert write(with_(write_args(), slots=tens(fq.DT_INT32, (T + 1,)))) == INVAL
    assert write(with_(write_args(), slots=tens(fq.DT_FLOAT32, (T,)))) == INVAL
    assert write(with_(write_args(), slots=tens(fq.DT_INT32, (T,), [2]))) == INVAL
    assert read(with_(read_args(), cu=tens(fq.DT_INT32, (B,)))) == INVAL
    assert read(with_(read_args(), bt=tens(fq.DT_INT32, (B, 2), [2, 2]))) == INVAL
    assert decode(with_(decode_args(), lens=tens(fq.DT_INT32, (B + 1,)))) == INVAL
    assert decode(with_(decode_args(), bt=tens(fq.DT_INT32, (B + 1, 2)))) == INVAL
    assert decode(with_(decode_args(), lse=tens(fq.DT_FLOAT32, (B, HQ + 1)))) == INVAL
    assert decode(with_(decode_args(), lse=tens(fq.DT_FLOAT16, (B, HQ)))) == INVAL
    assert prefill(with_(prefill_args(), ck=tens(fq.DT_INT32, (B,)))) == INVAL
    assert prefill(prefill_args(b=0)) == INVAL
    assert prefill(with_(prefill_args(), lse=tens(fq.DT_FLOAT32, (T, HQ), [1, T]))) == INVAL


def test_head_counts_refused():
    assert decode(with_(decode_args(), q=tens(fq.DT_BFLOAT16, (B, 3, D)), out=tens(fq.DT_BFLOAT16, (B, 3, D)))) == INVAL
    assert prefill(prefill_args(hq=3)) == INVAL
    assert prefill(prefill_args(d=260)) == INVAL
    assert prefill(prefill_args(d=12)) == INVAL
    wide = 2 ** 23 + 8  # elements between key rows
    assert prefill(with_(prefill_args(), k=tens(fq.DT_BFLOAT16, (T, H, D), [wide, D, 1]))) == INVAL


def test_a_16_bit_cache_takes_its_own_dtype_only():
    a = with_(write_args("f16"))
    assert write(a) == INVAL  # bf16 rows
    assert read(read_args("f16")) == INVAL
    assert decode(decode_args("f16")) == INVAL


def test_workspaces():
    size = ctypes.c_uint64(77)
    q = lambda a: fq.lib.fq_attn_decode_get_workspace_size(ref(a["q"]), ref(a["kc"]), ref(a["bt"]), ctypes.byref(size))  # noqa: E731
    assert q(decode_args()) == OK and size.value == 0  # a table of 32 tokens needs no join
    long = decode_args(width=64)
    assert q(long) == OK and size.value > 0
    need = size.value
    assert decode(long) == NULLP
    assert decode(with_(long, ws=DUMMY, size=need - 1)) == INVAL
    assert decode(with_(long, ws=DUMMY + 4, size=need)) == INVAL
    huge = dict(long, q=tens(fq.DT_BFLOAT16, (65536, HQ, D)), bt=tens(fq.DT_INT32, (65536, 2 ** 22)))
    assert q(huge) == INVAL  # more units of work than 31 bits count
    assert fq.lib.fq_attn_decode_get_workspace_size(None, ref(long["kc"]), ref(long["bt"]), ctypes.byref(size)) == NULLP
    assert fq.lib.fq_attn_decode_get_workspace_size(ref(long["q"]), ref(long["kc"]), ref(long["bt"]), None) == NULLP
    p = lambda a: fq.lib.fq_attn_prefill_get_workspace_size(ref(a["q"]), ref(a["k"]), ref(a["cq"]), a["causal"], ctypes.byref(size))  # noqa: E731
    assert p(prefill_args()) == OK and size.value == 0
    few = prefill_args(tk=8192)
    assert p(few) == OK and size.value > 0
    assert prefill(few) == NULLP
    assert prefill(with_(few, ws=DUMMY, size=size.value - 1)) == INVAL
    assert p(prefill_args(tq=65536, tk=65536)) == OK and size.value == 0  # rows enough to fill the device


def test_decode_reach_is_bounded():
    """A table whose reach a step past the last token could carry beyond 31 bits is refused."""
    size = ctypes.c_uint64()
    for width, want in ((2 ** 27 - 4096, INVAL), (2 ** 27, INVAL), (2 ** 26, OK)):
        a = decode_args(width=width)
        assert a["kc"].shape[2] == 16
        assert fq.lib.fq_attn_decode_get_workspace_size(ref(a["q"]), ref(a["kc"]), ref(a["bt"]), ctypes.byref(size)) == want
        if want == INVAL:
            assert decode(with_(a, ws=DUMMY, size=2 ** 40)) == INVAL


def test_python_arguments_refused():
    c = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        fq.KVCache("int3", c(2, 1, 16, 64), c(2, 1, 16, 64))
    with pytest.raises(ValueError):
        fq.KVCache("bf16", c(2, 1, 16, 64), c(2, 1, 16, 64))
    with pytest.raises(ValueError):
        fq.KVCache("int4", c(2, 1, 16, 32), c(2, 1, 16, 32))  # no scales
    with pytest.raises(ValueError):
        fq.KVCache("fp4", c(2, 1, 16, 32), c(2, 1, 16, 32), c(2, 1, 16, dt=torch.float32), c(2, 1, 16, dt=torch.float32))
    with pytest.raises(ValueError):
        fq.empty_kv_cache(2, 1, 16, 64, "e5m2", "cpu")
    cache = fq.empty_kv_cache(2, 3, 16, 64, "fp4", "cpu")
    assert cache.k.shape == (2, 3, 16, 32) and cache.k_scale.shape == (2, 3, 16, 2)
    assert (cache.pages, cache.heads, cache.page_size, cache.head_dim) == (2, 3, 16, 64)
    with pytest.raises(ValueError):
        fq.kv_read(cache, None, None, 5, torch.bfloat16, k_out=torch.empty(5, 3, 64))
