"""The Python side of the cache and attention calls (CPU only)."""
import ctypes

import pytest
import torch

import flatquant_transform_quant_amd as fq


def _desc(ptr):
    return fq.FqTensor.from_address(ptr)


@pytest.mark.parametrize("mode", fq.KV_MODES)
def test_a_cache_holds_on_to_its_tensors(mode):
    """The tensors of a handle cannot be exchanged under it: its calls would go on at the old addresses."""
    cache, other = (fq.empty_kv_cache(n, 2, 16, 64, mode, "cpu") for n in (4, 9))
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(other, name))
    assert cache.k.shape[0] == cache.pages == 4
    assert (cache.k_scale is None) == (mode in ("f16", "bf16"))


@pytest.mark.parametrize("mode", ["bf16", "int8", "fp4"])
def test_calls_follow_memory_that_has_moved(mode):
    """A cache tensor that is grown in place has other memory: descriptors and sizes are those of the moment."""
    cache = fq.empty_kv_cache(4, 2, 16, 64, mode, "cpu")
    before = [None if t is None else t.data_ptr() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.resize_(4096, *t.shape[1:])
    after = [None if t is None else t.data_ptr() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    assert all(a is None or a != b for a, b in zip(after, before))
    got = [None if p is None else (_desc(p).data, _desc(p).shape[0]) for p in cache._args()]
    assert got == [None if a is None else (a, 4096) for a in after]
    assert cache.pages == 4096
    assert cache._args() is cache._args()  # (nothing is built anew while they stay)


def test_memory_that_is_given_up_is_not_used():
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    cache.k.untyped_storage().resize_(0)
    size = ctypes.c_uint64()
    k = _desc(cache._args()[0])
    assert not k.data
    q, table, lens = torch.empty(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    d = fq._Descs(q, table, lens, q)
    assert fq.lib.fq_attn_decode(d.ptrs[0], *cache._args(), d.ptrs[1], d.ptrs[2], 0.0, d.ptrs[3], None, None, size, None) == fq.FQ_ERR_PARAM_NULLPTR


@pytest.fixture
def launches(monkeypatch):
    """Names of the launching calls of the library that the binding made; none is made in earnest."""
    made, real = [], fq.lib

    class Library:
        def __getattr__(self, name):
            if name in ("fq_kv_write", "fq_kv_read", "fq_attn_decode", "fq_attn_prefill", "fq_run", "fq_dequant", "fq_int4_gemm", "fq_mx_gemm"):
                return lambda *a: made.append(name) or fq.FQ_SUCCESS
            return getattr(real, name)

    monkeypatch.setattr(fq, "lib", Library())
    return made


class _Stream:
    cuda_stream = 0x1234

    def __init__(self, device="cuda:0"):
        self.device = torch.device(device)


def _calls(stream):
    """Every launching call of the package on host tensors."""
    b16, i32, u8, f32 = (lambda *s, t=t: torch.zeros(s, dtype=t) for t in (torch.bfloat16, torch.int32, torch.uint8, torch.float32))
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    rows, q, one, table = b16(3, 2, 64), b16(1, 4, 64), i32(1), i32(1, 2)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    out, sc = fq.empty_outputs(4, 64, 64, "int4", device="cpu")
    x, p = b16(4, 64, 64), b16(64, 64)
    return {
        "kv_write": lambda: fq.kv_write(cache, rows, rows, i32(3), stream=stream),
        "kv_read": lambda: fq.kv_read(cache, table, cu, 3, torch.bfloat16, rows, rows.clone(), stream=stream),
        "attn_decode": lambda: fq.attn_decode(q, cache, table, one, out=q.clone(), stream=stream),
        "attn_prefill": lambda: fq.attn_prefill(rows, rows, rows, cu, out=rows.clone(), stream=stream),
        "quantize": lambda: fq.quantize(x, p, p, out, sc, "int4", stream=stream),
        "dequantize": lambda: fq.dequantize(out, sc, "int4", 64, 64, torch.bfloat16, out=x.clone(), stream=stream),
        "int4_gemm": lambda: fq.int4_gemm(u8(4, 64), f32(4), u8(8, 64), f32(8), 128, out=b16(4, 8), stream=stream),
        "mx_gemm": lambda: fq.mx_gemm(u8(4, 64), u8(4, 2, 2), u8(8, 64), u8(8, 2, 2), 128, out=b16(4, 8), stream=stream),
    }


@pytest.mark.parametrize("name", list(_calls(None)))
def test_host_tensors_never_reach_a_launch(launches, name):
    """Also with a stream in hand, whose presence says nothing about where the tensors are."""
    with pytest.raises(ValueError, match="GPU"):
        _calls(_Stream())[name]()
    assert not launches


def test_a_stream_of_another_device_is_refused():
    class On:  # a tensor of cuda:0, as far as the check looks
        device = torch.device("cuda:0")

        def get_device(self):
            return 0

    fq._same_gpu(_Stream("cuda:0"), On(), None, On())
    with pytest.raises(ValueError, match="stream"):
        fq._same_gpu(_Stream("cuda:1"), On())


@pytest.fixture
def streams(monkeypatch):
    """A stand-in for torch's streams: two of them, the current one, and which was current at each allocation."""
    main, side, state = _Stream(), _Stream(), {"made": [], "recorded": []}
    state.update(main=main, side=side, current=main)

    class Inside:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, state["current"] = state["current"], self.s

        def __exit__(self, *_):
            state["current"] = self.before

    real = torch.empty, torch.empty_like

    def noted(f):
        def make(*a, **k):
            state["made"].append(state["current"])
            return f(*a, **k)
        return make

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["current"])
    monkeypatch.setattr(torch.cuda, "stream", Inside)
    monkeypatch.setattr(torch, "empty", noted(real[0]))
    monkeypatch.setattr(torch, "empty_like", noted(real[1]))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["recorded"].append((t.data_ptr(), s)))
    monkeypatch.setattr(fq, "_same_gpu", lambda *a: None)
    monkeypatch.setattr(fq, "_raw_stream", [lambda index: state["current"].cuda_stream])
    return state


def test_memory_of_a_call_comes_from_the_stream_it_runs_on(streams, launches):
    """Results and workspaces of a call on the caller's stream: a block of the current stream's pool may still be written by
    kernels that the caller's stream does not wait for."""
    main, side = streams["main"], streams["side"]
    b16, i32 = (lambda *s, t=t: torch.zeros(s, dtype=t) for t in (torch.bfloat16, torch.int32))
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    long = i32(1, 64)
    cq, ck = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([0, 8192], dtype=torch.int32)
    u8, f32 = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4)
    e8, made = torch.zeros(4, 2, 2, dtype=torch.uint8), streams["made"]

    def on(stream, count, results, f):
        made.clear()
        streams["recorded"].clear()
        f()
        assert made == [stream] * count and streams["current"] is main
        # (a result's memory waits for the current stream too when it is freed; a workspace's needs not)
        if results is not None:
            assert [s for _, s in streams["recorded"]] == ([main] * results if stream is side else [])

    for s, at in ((side, side), (None, main), (main, main)):
        on(at, 2, 2, lambda: fq.kv_read(cache, i32(1, 2), cq, 3, torch.bfloat16, stream=s))
        on(at, 2, 1, lambda: fq.attn_decode(b16(1, 4, 64), cache, long, i32(1), stream=s))
        on(at, 2, 1, lambda: fq.attn_prefill(b16(3, 4, 64), b16(8192, 2, 64), b16(8192, 2, 64), cq, ck, stream=s))
        on(at, 1, 1, lambda: fq.dequantize(torch.zeros(4, 64, 32, dtype=torch.uint8), f32, "int4", 64, 64, torch.bfloat16, stream=s))
        on(at, 1, 1, lambda: fq.int4_gemm(u8, f32, u8, f32, 128, stream=s))
        on(at, 1, 1, lambda: fq.mx_gemm(u8, e8, u8, e8, 128, stream=s))
        x, p = b16(4, 256, 256), b16(256, 256)
        out, sc = fq.empty_outputs(4, 256, 256, "int4", device="cpu")
        on(at, 1, None, lambda: fq.quantize(x, p, p, out, sc, "int4", 0.95, stream=s))
    assert launches.count("fq_attn_decode") == 3


def test_a_workspace_is_contiguous(streams, launches):
    """One whose elements lie over each other has less memory than it has elements, one with gaps more."""
    b16, i32 = (lambda *s, t=t: torch.zeros(s, dtype=t) for t in (torch.bfloat16, torch.int32))
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    q, table, lens = b16(1, 4, 64), i32(1, 64), i32(1)
    size = fq.attn_decode_workspace_size(q, cache, table)
    assert size > 0
    cu, ck = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([0, 8192], dtype=torch.int32)
    k = b16(8192, 2, 64)
    more = fq.attn_prefill_workspace_size(b16(3, 4, 64), k, cu)
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(max(size, more)), torch.zeros(2 * max(size, more), dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            fq.attn_decode(q, cache, table, lens, workspace=bad)
        with pytest.raises(ValueError, match="contiguous"):
            fq.attn_prefill(b16(3, 4, 64), k, k, cu, ck, workspace=bad)
    assert not launches
    fq.attn_decode(q, cache, table, lens, workspace=torch.zeros(size, dtype=torch.uint8))
    assert launches == ["fq_attn_decode"]
