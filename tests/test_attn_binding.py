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
