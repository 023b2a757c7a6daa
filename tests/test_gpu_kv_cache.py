"""GPU: the paged cache.  Codes, scales and values read back are compared bit for bit with the
plain encoder (IEEE fp32 quotients, explicit tables): every step has one defined result."""
import math

import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, encode, pack, values
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
LOW = ["int8", "e4m3", "int4", "fp4"]


def _rows(T, H, D, dt, seed):
    """Rows over many magnitudes, with zeros, ties, subnormals, and rows that hold an infinity or a NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(torch.empty(T, H, 1).uniform_(-8, 8, generator=g))
    x = x.to(TDT[dt])
    f = x.view(T * H, D)
    n = T * H
    f[1 % n] = 0.0
    f[2 % n] = torch.tensor([7.0, 3.5, -3.5, 0.5, -0.5, 1.5, 2.5, -7.0] * (D // 8)).to(f.dtype)
    f[3 % n] = (127.0 * torch.tensor([1.0, 0.5, -0.5, 0.25, 0.125, -1.0, 0.75, -0.0] * (D // 8))).to(f.dtype)
    f[4 % n] = f[4 % n] * (1e-30 if dt == "bf16" else 1e-5)
    f[5 % n] = (1e-39 if dt == "bf16" else 6e-8) * torch.ones(D)
    f[6 % n, D // 2] = math.inf
    f[7 % n, D - 1] = math.nan
    f[8 % n, 0] = -math.inf
    return x


def _host(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _place(cache, codes, scales, slots, T, H):
    """The rows that slots name, gathered from the cache on the host."""
    P = cache.page_size
    c, s = _host(codes), None if scales is None else scales.cpu().numpy()
    rows = np.stack([c[sl // P, :, sl % P] for sl in slots])
    return rows, None if s is None else np.stack([s[sl // P, :, sl % P] for sl in slots])


def _slots(T, pages, P, seed):
    return np.random.default_rng(seed).permutation(pages * P)[:T].astype(np.int32)


@pytest.mark.parametrize("mode", LOW + ["same"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (33, 3, 128, 16), (70, 8, 96, 64), (19, 2, 256, 32), (257, 5, 32, 1024), (40, 1, 160, 16)])
def test_write_then_read(mode, dt, T, H, D, P):
    m = dt if mode == "same" else mode
    say(f"[gpu] kv {m} {dt} T={T} H={H} D={D} P={P}")
    pages = -(-T // P) + 2
    k, v = _rows(T, H, D, dt, 1), _rows(T, H, D, dt, 2).flip(0).contiguous()
    slots = _slots(T, pages, P, 3)
    cache = fq.empty_kv_cache(pages, H, P, D, m, DEV)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0xAA)
    fq.kv_write(cache, k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV))
    # read back in order: a table and positions cannot name scattered slots, so gather on the host
    untouched = np.ones(pages * P, bool)
    untouched[slots] = False
    for x, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        got, gs = _place(cache, codes, scales, slots, T, H)
        if mode == "same":
            assert (got == x.view(torch.uint8).numpy()).all()
        else:
            code, want_s = encode(x, mode)
            assert (got == pack(code, mode)).all(), np.argwhere(got != pack(code, mode))[:4].tolist()
            if mode == "fp4":
                assert (gs == want_s).all()
            else:
                assert (gs.view(np.uint32) == want_s.view(np.uint32)).all() or (
                    np.isnan(gs) == np.isnan(want_s)).all() and (gs[~np.isnan(gs)] == want_s[~np.isnan(want_s)]).all()
        raw = _host(codes).transpose(0, 2, 1, 3).reshape(pages * P, -1)
        assert (raw[untouched] == 0xAA).all()
    # sequences read back through a table: tokens in slot order
    lens = [pages * P, 0, 5, P + 1 if pages > 1 else P]
    table = np.full((4, pages), -1, np.int32)
    perm = np.random.default_rng(4).permutation(pages)
    table[0] = perm
    table[2, 0], table[3, :2] = perm[0], perm[1:3]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = int(cu[-1])
    ko, vo = fq.kv_read(cache, torch.from_numpy(table).to(DEV), torch.from_numpy(cu).to(DEV), total, TDT[dt])
    written = np.zeros(pages * P, bool)
    written[slots] = True
    for x, out in ((k, ko), (v, vo)):
        if mode == "same":
            ref = x
        else:
            with np.errstate(over="ignore"):
                ref = torch.from_numpy(values(*encode(x, mode), mode)).float().to(TDT[dt])
        where = {int(s): i for i, s in enumerate(slots)}
        out = out.cpu()
        r = 0
        for b, n in enumerate(lens):
            for t in range(n):
                sl = int(table[b, t // P]) * P + t % P
                if written[sl]:
                    a, w = out[r], ref[where[sl]]
                    same = (a.view(torch.int16) == w.view(torch.int16)) | (a.isnan() & w.isnan())
                    assert same.all(), (b, t, mode, dt)
                r += 1


@pytest.mark.parametrize("mode,clip,dmax", [("int8", 0.9, 0.0), ("int4", 0.8, 0.0), ("e4m3", 0.5, 0.0), ("fp4", 1.0, 6.0),
                                            ("fp4", 1.0, 8.0), ("fp4", 1.0, 12.0), ("int4", 1e-6, 0.0)])
def test_clip_and_type_max(mode, clip, dmax):
    T, H, D, P = 48, 4, 128, 16
    x = _rows(T, H, D, "bf16", 7)
    slots = np.arange(T, dtype=np.int32)
    cache = fq.empty_kv_cache(3, H, P, D, mode, DEV)
    fq.kv_write(cache, x.to(DEV), x.to(DEV), torch.from_numpy(slots).to(DEV), clip, dmax)
    code, sc = encode(x, mode, clip, dmax)
    got, gs = _place(cache, cache.v, cache.v_scale, slots, T, H)
    assert (got == pack(code, mode)).all()
    assert np.array_equal(gs, sc.astype(gs.dtype), equal_nan=mode != "fp4")


@pytest.mark.parametrize("mode", LOW + ["bf16"])
def test_slots_outside_the_cache_write_nothing(mode):
    H, P, D = 2, 16, 64
    cache = fq.empty_kv_cache(2, H, P, D, mode, DEV)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0x55)
    slots = torch.tensor([-1, 2 * P, 2 ** 31 - 1, -2 ** 31, 3], dtype=torch.int32, device=DEV)
    x = torch.ones(5, H, D, dtype=torch.bfloat16, device=DEV)
    fq.kv_write(cache, x, x, slots)
    raw = _host(cache.k).transpose(0, 2, 1, 3).reshape(2 * P, -1)
    keep = np.arange(2 * P) != 3
    assert (raw[keep] == 0x55).all() and not (raw[3] == 0x55).all()
    # and reading a table entry outside the cache gives zeros
    table = torch.tensor([[5, 0], [-3, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20, 40 + 8], dtype=torch.int32, device=DEV)
    k, v = (torch.full((50, H, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fq.kv_read(cache, table, cu, 50, torch.bfloat16, k, v)
    for t in (k, v):
        assert (t[:16] == 0).all() and (t[20:48] == 0).all() and (t[48:] == 9.0).all()
    assert (k[19] == 1.0).all()  # position 19 = page 0, offset 3


@pytest.mark.parametrize("mode", LOW + ["f16"])
def test_strided_rows_and_interleaved_cache(mode):
    """Rows cut from one fused projection; both sides' pages interleaved in one allocation; outputs into a wider buffer."""
    T, Hq, H, D, P, pages = 37, 6, 2, 64, 16, 4
    qkv = torch.randn(T, Hq + 2 * H, D, generator=torch.Generator().manual_seed(3)).half().to(DEV)
    k, v = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    ref = fq.empty_kv_cache(pages, H, P, D, mode, DEV)
    both = torch.stack([ref.k, ref.v], 1).view(torch.uint8).fill_(0).view(ref.k.dtype)
    sc = None if ref.k_scale is None else torch.stack([ref.k_scale, ref.v_scale], 1)
    cache = fq.KVCache(mode, both[:, 0], both[:, 1], *((None, None) if sc is None else (sc[:, 0], sc[:, 1])))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    fq.kv_write(cache, k, v, slots)
    fq.kv_write(ref, k.contiguous(), v.contiguous(), slots)
    n = 2 * P
    assert torch.equal(cache.k[:2].contiguous().view(torch.uint8), ref.k[:2].contiguous().view(torch.uint8))
    assert torch.equal(cache.v[:2].contiguous().view(torch.uint8), ref.v[:2].contiguous().view(torch.uint8))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None].expand(1, pages)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    wide = torch.zeros(n, 2 * H + 1, D, dtype=torch.float16, device=DEV)
    fq.kv_read(cache, table, cu, n, torch.float16, wide[:, :H], wide[:, H:2 * H])
    a, b = fq.kv_read(ref, table, cu, n, torch.float16)
    assert torch.equal(wide[:, :H], a) and torch.equal(wide[:, H:2 * H], b) and (wide[:, 2 * H] == 0).all()


def test_nothing_to_do():
    cache = fq.empty_kv_cache(2, 2, 16, 64, "int8", DEV)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    fq.kv_write(cache, e, e, torch.empty(0, dtype=torch.int32, device=DEV))
    k, v = fq.kv_read(cache, torch.empty(0, 3, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), 0, torch.bfloat16)
    assert k.shape == v.shape == (0, 2, 64)
    # sequences of length 0 only, and a table without columns
    k, v = fq.kv_read(cache, torch.empty(3, 0, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV), 0, torch.bfloat16)
    torch.cuda.synchronize()
    assert k.numel() == 0


def test_offsets_past_32_bits():
    """A cache side of 4.5 GB: the last page lies past 2^32 bytes."""
    H, P, D = 8, 1024, 256
    pages = 2304  # 8 * 1024 * 256 bytes = 2 MB a page
    cache = fq.empty_kv_cache(pages, H, P, D, "int8", DEV)
    x = _rows(40, H, D, "bf16", 5)
    slots = np.concatenate([np.arange(20), np.arange(20) + (pages - 1) * P + 7]).astype(np.int32)
    fq.kv_write(cache, x.to(DEV), x.to(DEV), torch.from_numpy(slots).to(DEV))
    code, sc = encode(x, "int8")
    got = cache.v[pages - 1, :, 7:27].view(torch.uint8).cpu().numpy().transpose(1, 0, 2)
    assert (got == pack(code, "int8")[20:]).all()
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    k, v = fq.kv_read(cache, table, torch.tensor([0, 27], dtype=torch.int32, device=DEV), 27, torch.bfloat16)
    want = torch.from_numpy(values(code[20:], sc[20:], "int8")).float().bfloat16()
    got = k[7:27].cpu()
    assert ((got == want) | (got.isnan() & want.isnan())).all()
