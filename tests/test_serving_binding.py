"""The Python side of rotation, append, attention of new tokens and the int8 product (CPU only)."""
import pytest
import torch

import flatquant_transform_quant_amd as fq
from test_attn_binding import _Stream, streams  # noqa: F401

NAMES = ("fq_qk_rope", "fq_kv_append", "fq_attn_chunk", "fq_int8_gemm")


@pytest.fixture
def launches(monkeypatch):
    made, real = [], fq.lib

    class Library:
        def __getattr__(self, name):
            return (lambda *a: made.append(name) or fq.FQ_SUCCESS) if name in NAMES else getattr(real, name)

    monkeypatch.setattr(fq, "lib", Library())
    return made


def _b16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def _calls(stream, given=True):
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    q, k, freq, cu = _b16(3, 4, 64), _b16(3, 2, 64), torch.zeros(32), torch.tensor([0, 3], dtype=torch.int32)
    a = torch.zeros(3, 256, dtype=torch.int8), torch.zeros(3), torch.zeros(8, 256, dtype=torch.int8), torch.zeros(8)
    out = (lambda t: t.clone()) if given else (lambda t: None)
    return {
        "qk_rope": lambda: fq.qk_rope(q, k, _i32(3), freq, q_out=out(q), k_out=out(k), stream=stream),
        "kv_append": lambda: fq.kv_append(cache, q, k, k, _i32(3), _i32(3), freq, q_out=out(q), stream=stream),
        "attn_chunk": lambda: fq.attn_chunk(q, cache, _i32(1, 200), cu, _i32(1), out=out(q), stream=stream),
        "int8_gemm": lambda: fq.int8_gemm(*a, out=out(_b16(3, 8)), stream=stream),
    }


@pytest.mark.parametrize("stream", [None, _Stream()], ids=["current", "given"])
@pytest.mark.parametrize("name", list(_calls(None)))
def test_host_tensors_never_reach_a_launch(launches, name, stream):
    with pytest.raises(ValueError, match="GPU"):
        _calls(stream)[name]()
    assert not launches


@pytest.mark.parametrize("name,blocks,results", [("qk_rope", 2, 2), ("kv_append", 1, 1), ("attn_chunk", 2, 1), ("int8_gemm", 1, 1)])
def test_memory_of_a_call_comes_from_the_stream_it_runs_on(streams, launches, name, blocks, results):  # noqa: F811
    main, side = streams["main"], streams["side"]
    for s, at in ((side, side), (None, main), (main, main)):
        call = _calls(s, given=False)[name]
        streams["made"].clear()
        streams["recorded"].clear()
        call()
        assert streams["made"] == [at] * blocks and streams["current"] is main
        assert [r for _, r in streams["recorded"]] == ([main] * results if at is side else [])
    assert launches == ["fq_" + name] * 3


def test_a_workspace_is_contiguous(streams, launches):  # noqa: F811
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    q, table, cu, lens = _b16(3, 4, 64), _i32(1, 200), torch.tensor([0, 3], dtype=torch.int32), _i32(1)
    size = fq.attn_chunk_workspace_size(q, cache, table, cu)
    assert size > 0
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(size), torch.zeros(2 * size, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            fq.attn_chunk(q, cache, table, cu, lens, workspace=bad)
    assert not launches
    fq.attn_chunk(q, cache, table, cu, lens, workspace=torch.zeros(size, dtype=torch.uint8))
    assert launches == ["fq_attn_chunk"]


@pytest.mark.parametrize("window,sinks,same", [(2 ** 32 + 5, 0, (0, 0)), (2 ** 40, 2 ** 32, (0, 0)), (100, 2 ** 32 + 1, (100, 2 ** 31 - 1))])
def test_windows_past_32_bits(window, sinks, same):
    """A window beyond every length is none; its low bits are not taken for a short one."""
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    at = _b16(3, 4, 64), cache, _i32(1, 4096), torch.tensor([0, 3], dtype=torch.int32)
    want = fq.attn_chunk_workspace_size(*at, *same)
    assert want > 0 and fq.attn_chunk_workspace_size(*at, window, sinks) == want


@pytest.mark.parametrize("window,sinks", [(-1, 0), (-2 ** 32 + 5, 0), (100, -2 ** 32 + 5)])
def test_lengths_below_zero_are_refused(window, sinks):
    cache = fq.empty_kv_cache(4, 2, 16, 64, "int8", "cpu")
    with pytest.raises(fq.FqError):
        fq.attn_chunk_workspace_size(_b16(3, 4, 64), cache, _i32(1, 4096), torch.tensor([0, 3], dtype=torch.int32), window, sinks)
