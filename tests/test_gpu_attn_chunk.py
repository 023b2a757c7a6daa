"""GPU: attention of new tokens over the paged cache, with and without a window, against fp64 with the derived
elementwise bound of attn_ref.bound."""
import math

import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, U
from gpu_util import DEV, say
from test_gpu_attention import MODES, _check_rows, _fill

pytestmark = pytest.mark.gpu


def seen_by(Lq, Lk, window, sinks):
    """[Lq, Lk]: the keys that each row sees."""
    at, j = torch.arange(Lk - Lq, Lk)[:, None], torch.arange(Lk)[None]
    ok = j <= at
    if window:
        ok &= (j > at - window) | (j < sinks)
    return ok


def attend(q, k, v, seen, scale):
    """One sequence in fp64 (as attn_ref.softmax_attend, any visibility)."""
    Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[:2]
    if Lk == 0 or Lq == 0:
        z = torch.zeros(Lq, Hq, D, dtype=torch.float64)
        return z, torch.full((Lq, Hq), -math.inf, dtype=torch.float64), z, z[..., 0], torch.zeros(Hq, D, dtype=torch.float64)
    some = seen.any(0)[:, None, None]
    kk, vv = (torch.where(some, t, 0.0).repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for t in (k, v))
    qq = q.transpose(0, 1)
    s, mass = (qq @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf), (qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)).masked_fill(~seen, 0.0)
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    return (p @ vv).transpose(0, 1), lse.T, (p @ vv.abs()).transpose(0, 1), mass.amax(-1).T, vv.abs().amax(1)


def _run(sizes, Hq, H, D, P, mode, dt, window=0, sinks=0, seed=0, scale=0.0, dead=(), wide=0):
    """sizes: (new rows, cached tokens) of each sequence; `dead`: (sequence, page) entries that are taken out of the table."""
    lens = [n for _, n in sizes]
    cache, table, ks, vs = _fill(lens, H, D, P, mode, dt, seed)
    for b, i in dead:
        table[b, i] = -1 if (b + i) % 2 else cache.pages
    cu = np.concatenate([[0], np.cumsum([r for r, _ in sizes])]).astype(np.int32)
    T, extra = int(cu[-1]), 3
    g = torch.Generator().manual_seed(seed + 1)
    # queries out of a wider tensor, and rows behind the last sequence
    q = (2.0 * torch.randn(T + extra, Hq + wide, D, generator=g)).to(TDT[dt])
    qd = q.to(DEV)[:, :Hq]
    out = torch.full((T + extra, Hq, D), 7.0, dtype=TDT[dt], device=DEV)
    lse = torch.full((T + extra, Hq), 7.0, device=DEV)
    got = fq.attn_chunk(qd, cache, table, torch.from_numpy(cu).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), window, sinks, scale, out, lse)
    torch.cuda.synchronize()
    assert got is out and (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()
    again = fq.attn_chunk(qd, cache, table, torch.from_numpy(cu).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), window, sinks, scale)
    assert torch.equal(again[:T], out[:T])
    out, lse = out.cpu(), lse.cpu()
    for b, (r, n) in enumerate(sizes):
        seen = seen_by(r, n, window, sinks)
        for bb, i in dead:
            if bb == b:
                seen[:, i * P:(i + 1) * P] = False
        want = attend(q[cu[b]:cu[b + 1], :Hq].double(), ks[b], vs[b], seen, scale or 1 / math.sqrt(D))
        _check_rows(out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], want, dt, D, n, dt if mode == "same" else "f16", f"b={b} rows={r} keys={n}")


SIZES = [(1, 1), (3, 0), (0, 40), (1, 17), (5, 64), (2, 65), (4, 3), (33, 130), (64, 64), (20, 300)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,H,D,P", [(4, 4, 64, 16), (8, 1, 128, 32), (14, 2, 96, 16), (3, 3, 256, 64), (20, 1, 128, 128), (16, 2, 32, 16), (5, 1, 160, 16)])
def test_chunk(mode, dt, Hq, H, D, P):
    say(f"[gpu] chunk {mode} {dt} Hq={Hq} H={H} D={D} P={P}")
    _run(SIZES, Hq, H, D, P, mode, dt)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,P", [(64, 16), (96, 32), (128, 16), (256, 16)])
@pytest.mark.parametrize("rows", [1, 3, 6])
def test_row_tiles(mode, D, P, rows):
    """Row tiles of 32, 64 and 128 (by the mean number of rows of a cache head: 16, 48 and 96), sequences of other numbers among them,
    some long enough that their walks are split."""
    for window, sinks in ((0, 0), (300, 20)):
        say(f"[gpu] tiles {mode} D={D} rows={rows} window={window}")
        _run([(rows, 2100), (2 * rows, 70), (rows, 15), (0, 33), (1, 901)], 16, 1, D, P, mode, "bf16", window, sinks, seed=20)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 300), (37, 4), (64, 64), (65, 0), (128, 65), (100000, 7)])
def test_window(mode, window, sinks):
    for Hq, H, D, P, dt in ((8, 2, 64, 16, "bf16"), (7, 1, 128, 32, "f16")):
        say(f"[gpu] window {window} sinks {sinks} {mode} {dt} Hq={Hq} H={H} D={D} P={P}")
        _run(SIZES + [(70, 700)], Hq, H, D, P, mode, dt, window, sinks, seed=2)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("Hq,H,D,P", [(8, 1, 128, 64), (6, 2, 64, 16), (4, 1, 256, 32), (3, 3, 96, 16)])
def test_long_walks_are_split(mode, Hq, H, D, P):
    """Few rows over many keys: runs that hold parts of a segment, one and several of them; windows far from the start."""
    for window, sinks in ((0, 0), (1500, 70)):
        say(f"[gpu] long {mode} Hq={Hq} H={H} D={D} window={window}")
        _run([(2, 5000), (1, 1), (0, 0), (40, 2500), (3, 777)], Hq, H, D, P, mode, "bf16", window, sinks, seed=3)


@pytest.mark.parametrize("mode", ["same", "int8", "fp4"])
def test_many_sequences(mode):
    """More than a wave plans at once, idle places among them."""
    sizes = [((i * i) % 4, (37 * i) % 400) for i in range(150)]
    for window, sinks in ((0, 0), (50, 5)):
        say(f"[gpu] many {mode} window={window}")
        _run(sizes, 4, 2, 64, 16, mode, "f16", window, sinks, seed=4)


@pytest.mark.parametrize("mode", ["same", "int8", "fp4"])
def test_many_sequences_dealt(mode):
    """The same with long ones among them, so that the work is dealt in runs over many short segments and parts of long ones."""
    sizes = [((i * i) % 4, (37 * i) % 400) for i in range(70)] + [(2, 3000)] + [((i * i) % 7, (41 * i) % 300) for i in range(70)] + [(30, 1800)]
    for window, sinks in ((0, 0), (1700, 5)):
        say(f"[gpu] many dealt {mode} window={window}")
        _run(sizes, 4, 2, 64, 16, mode, "f16", window, sinks, seed=21)


@pytest.mark.parametrize("Hq,H", [(128, 1), (130, 1), (300, 1), (258, 2)])
def test_many_heads_on_one(Hq, H):
    """Up to 128 heads of a cache head are rows of one tile; more take several."""
    for mode in ("same", "int4"):
        say(f"[gpu] heads {Hq} on {H} {mode}")
        _run([(3, 90), (1, 5), (2, 700)], Hq, H, 64, 16, mode, "bf16", seed=5, wide=2)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 24, 40, 112, 200])
def test_odd_head_sizes(dt, D):
    for mode in ("same", "int8", "int4", "e4m3"):
        say(f"[gpu] chunk {mode} {dt} D={D}")
        _run([(1, 1), (9, 17), (3, 130)], 6, 2, D, 16, mode, dt, seed=6, wide=1)


@pytest.mark.parametrize("scale", [0.5, 4.0, -0.2, 1e-50])
def test_scales(scale):
    for mode in ("same", "e4m3", "fp4"):
        _run([(2, 40), (5, 700)], 8, 2, 64, 16, mode, "f16", seed=7, scale=scale)


@pytest.mark.parametrize("mode", MODES)
def test_pages_that_are_missing(mode):
    """Entries outside the cache: their tokens are left out, whole tiles of them, and a row that has no other gives zeros."""
    for P, dead in ((16, [(0, 0), (0, 3), (1, 5), (1, 6), (1, 7), (1, 8), (2, 0)]), (64, [(0, 1), (2, 0), (1, 2)])):
        say(f"[gpu] missing {mode} P={P}")
        _run([(5, 130), (2, 300), (3, 9)], 4, 2, 64, P, mode, "bf16", seed=8, dead=dead)


def _one(k, v, mode, P=16, spare=0):
    n, H, D = k.shape
    pages = -(-n // P)
    cache = fq.empty_kv_cache(pages + spare, H, P, D, mode, DEV)
    fq.kv_write(cache, k.to(DEV), v.to(DEV), torch.arange(n, dtype=torch.int32, device=DEV))
    return cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None]


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_infinities_in_16_bits(dt):
    """Infinities and NaN in keys and values reach the rows that see them, and no other; a seen infinity of a value stays one."""
    g = torch.Generator().manual_seed(9)
    n, r, Hq, H, D = 200, 120, 4, 2, 64
    q, k, v = (torch.randn(m, h, D, generator=g).to(TDT[dt]) for m, h in ((r, Hq), (n, H), (n, H)))
    v[150, 0, 7], v[190, 1, 9], k[180, 1, 3] = math.inf, math.nan, math.nan
    k[170, 0], v[170, 0, 11] = -30.0 * q[95, 0], -math.inf  # a weight that rounds to 0
    for window, sinks in ((0, 0), (25, 3)):
        say(f"[gpu] infinities {dt} window={window}")
        cache, table = _one(k, v, dt)
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), window, sinks).cpu().double()
        seen = seen_by(r, n, window, sinks)
        clean_k, clean_v = torch.where(torch.isfinite(k), k, 0.0).double(), torch.where(torch.isfinite(v), v, 0.0).double()
        out, _, absv, top, vmax = attend(q.double(), clean_k, clean_v, seen, 1 / math.sqrt(D))
        want = out.clone()
        for j, h, d, x in ((150, 0, 7, math.inf), (170, 0, 11, -math.inf), (190, 1, 9, math.nan)):
            want[seen[:, j], 2 * h:2 * h + 2, d] = x
        want[seen[:, 180], 2:4] = math.nan
        fin = torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~fin & ~want.isnan()], want[~fin & ~want.isnan()])
        from attn_ref import bound
        assert ((got - out).abs() <= bound(out, absv, top, vmax, n, D, dt, dt))[fin].all()


@pytest.mark.parametrize("mode", ["int8", "e4m3", "int4", "fp4"])
def test_rows_that_are_not_finite_in_low_bits(mode):
    """A cached row (E2M1: a group) that reads back as NaN makes NaN of the rows that see it, and only of those."""
    g = torch.Generator().manual_seed(10)
    n, r, Hq, H, D = 200, 120, 4, 2, 64
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, Hq), (n, H), (n, H)))
    k[180, 1, 3], v[150, 0, 40] = math.nan, math.inf
    clean = _one(torch.where(torch.isfinite(k), k, 0.0), torch.where(torch.isfinite(v), v, 0.0), mode)
    cache, table = _one(k, v, mode)
    for window, sinks in ((0, 0), (25, 3)):
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), window, sinks).cpu()
        ok = fq.attn_chunk(q.to(DEV), *clean, _i32(0, r), _i32(n), window, sinks).cpu()
        seen = seen_by(r, n, window, sinks)
        bad = torch.zeros(r, Hq, D, dtype=torch.bool)
        bad[seen[:, 180], 2:] = True
        bad[seen[:, 150], :2, 32 if mode == "fp4" else 0:] = True
        assert torch.equal(torch.isnan(got), bad)
        assert torch.equal(got[:30], ok[:30])  # (rows before both)


@pytest.mark.parametrize("mode", ["int8", "e4m3", "int4", "fp4"])
def test_hidden_values_of_any_size(mode):
    """A token that a row does not see does not cost the row's weights any bits, however large its values: the same cache
    with ordinary values there gives the same rows."""
    g = torch.Generator().manual_seed(11)
    n, r, Hq, H, D = 150, 100, 4, 2, 64
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, Hq), (n, H), (n, H)))
    big = v.clone()
    big[120] *= 2.0 ** 80
    for window, sinks in ((0, 0), (10, 3)):
        a, b = (fq.attn_chunk(q.to(DEV), *_one(k, x, mode), _i32(0, r), _i32(n), window, sinks).cpu() for x in (v, big))
        see = seen_by(r, n, window, sinks)[:, 120]
        # a row's reference moves with the scales it has seen: the sums' roundings may differ, the weights' bits not
        assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs() + 2.0 ** -9)[~see].all()
        assert (b.double().abs().amax(-1) > 2.0 ** 40)[see][:, :].any()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("e", [-70, -30, 30, 85])
def test_values_of_any_size(mode, e):
    """Values 2^e times as large give 2^e times the result: in 16 bits bit for bit, as the weights are the same numbers.  In the
    low-bit formats the reference R is part of the exponent that a weight is formed from, whose size is below 2^8 (|R| <= 120, a lead
    of 13): its rounding, 2^-17 at the most, moves a weight by 2^-17 ln 2 of itself and may move its rounding to 11 bits to the
    other neighbour, 2^-10 of itself.  Two such sets of weights give sums that differ by 2^-10 + 2^-16 of sum p |v| at most,
    and the outputs' own roundings may go to either side."""
    g = torch.Generator().manual_seed(12)
    n, r, Hq, H, D = 300, 7, 8, 2, 64
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, Hq), (n, H), (n, H)))
    m = "bf16" if mode == "same" else mode
    a, b = (fq.attn_chunk(q.to(DEV), *_one(k, x, m), _i32(0, r), _i32(n)).cpu() for x in (v, (v.double() * 2.0 ** e).bfloat16()))
    if mode == "same":
        assert torch.equal((a.double() * 2.0 ** e).bfloat16(), b)
        return
    cache, table = _one(k, v, m)
    kk, vv = (x.cpu().double() for x in fq.kv_read(cache, table, _i32(0, n), n, torch.bfloat16))
    absv = attend(q.double(), kk, vv, seen_by(r, n, 0, 0), 1 / math.sqrt(D))[2]
    # (the values as read back, and weights of keys as read back: each off by 2^-8, well within the factor 1.1)
    assert ((a.double() - b.double() * 2.0 ** -e).abs() <= 2.0 ** -7 * a.double().abs() + 1.1 * (2.0 ** -10 + 2.0 ** -16) * absv).all()


def test_rows_of_queries_and_outputs_anywhere():
    """Strides of queries and outputs, sequences whose rows are not all of a tile."""
    g = torch.Generator().manual_seed(13)
    n, Hq, H, D = 90, 6, 3, 64
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    cache, table = _one(k, v, "bf16")
    q = torch.randn(Hq, 11, D + 8, generator=g).bfloat16().to(DEV)  # heads outermost
    out = torch.zeros(11, 2 * Hq, D, dtype=torch.bfloat16, device=DEV)
    view = q.transpose(0, 1)[..., :D]
    fq.attn_chunk(view, cache, table, _i32(0, 11), _i32(n), out=out[:, Hq:])
    assert torch.equal(out[:, Hq:], fq.attn_chunk(view.contiguous(), cache, table, _i32(0, 11), _i32(n))) and (out[:, :Hq] == 0).all()


@pytest.mark.parametrize("mode", MODES)
def test_single_tokens_agree_with_decode(mode):
    """One new token a sequence and no window is fq_attn_decode's call: both within their own roundings of the same sums."""
    lens = [1, 700, 64, 0, 129]
    for dt in ("bf16", "f16"):
        cache, table, _, vs = _fill(lens, 2, 128, 16, mode, dt, 14)
        q = torch.randn(len(lens), 8, 128, generator=torch.Generator().manual_seed(1)).to(TDT[dt]).to(DEV)
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        a = fq.attn_decode(q, cache, table, n).cpu().double()
        b = fq.attn_chunk(q, cache, table, torch.arange(len(lens) + 1, dtype=torch.int32, device=DEV), n).cpu().double()
        for i, m in enumerate(lens):
            top = vs[i].abs().max() if m else 0.0
            assert ((a[i] - b[i]).abs() <= 2 * U[dt] * a[i].abs() + (U[dt] + 2.0 ** -18) * top).all()


def test_nothing_to_do():
    cache = fq.empty_kv_cache(2, 2, 16, 64, "int8", DEV)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert fq.attn_chunk(q, cache, _i32(0)[None], _i32(0, 0), _i32(5)).shape == (0, 4, 64)
    # a table without a column, and lengths past the table's reach or below zero
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, 4, device=DEV)
    out = fq.attn_chunk(q, cache, torch.empty(1, 0, dtype=torch.int32, device=DEV), _i32(0, 3), _i32(5), lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert (fq.attn_chunk(q, cache, _i32(0)[None], _i32(0, 3), _i32(-9)) == 0).all()
    cache.k.zero_(), cache.v.zero_(), cache.k_scale.fill_(1.0), cache.v_scale.fill_(1.0)
    assert torch.equal(fq.attn_chunk(q, cache, _i32(0)[None], _i32(0, 3), _i32(10 ** 6)), fq.attn_chunk(q, cache, _i32(0)[None], _i32(0, 3), _i32(16)))


@pytest.mark.parametrize("mode", ["bf16", "int8"])
def test_captured(mode):
    """A captured call replayed with other queries, lengths and pages, eager work in between, against eager calls."""
    g = torch.Generator().manual_seed(15)
    n, Hq, H, D, B = 2000, 8, 1, 128, 3
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    cache, _ = _one(k, v, mode)
    table = torch.stack([torch.randperm(cache.pages, generator=g) for _ in range(B)]).int().to(DEV)
    q = torch.randn(12, Hq, D, generator=g).bfloat16().to(DEV)
    cu, lens = _i32(0, 1, 6, 12), _i32(2000, 40, 1500)
    fq.attn_chunk(q, cache, table, cu, lens, 700, 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.attn_chunk(q, cache, table, cu, lens, 700, 5)
    for i in range(4):
        q.copy_(torch.randn(12, Hq, D, generator=g).bfloat16())
        cu.copy_(_i32(0, i, 7 + i, 12))
        lens.copy_(_i32(100 * i, 2000 - i, 900 + i))
        table.copy_(table.flip(0))
        want = fq.attn_chunk(q, cache, table, cu, lens, 700, 5)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_own_workspace_and_another_stream():
    g = torch.Generator().manual_seed(16)
    n, Hq, H, D = 3000, 8, 2, 128
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    cache, table = _one(k, v, "int4")
    q, cu, lens = torch.randn(5, Hq, D, generator=g).bfloat16().to(DEV), _i32(0, 5), _i32(n)
    want = fq.attn_chunk(q, cache, table, cu, lens)
    size = fq.attn_chunk_workspace_size(q, cache, table, cu)
    assert size > 0
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(fq.attn_chunk(q, cache, table, cu, lens, workspace=ws), want)
    with pytest.raises(fq.FqError):
        fq.attn_chunk(q, cache, table, cu, lens, workspace=ws[:-16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fq.attn_chunk(q, cache, table, cu, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("mode", ["bf16", "int8", "fp4"])
def test_pages_past_32_bits(mode):
    """Pages whose bytes lie past 2^32 of the cache's start."""
    H, P, D = 8, 128, 128
    per = H * P * D * (2 if mode == "bf16" else 1 if mode == "int8" else 0.5)
    pages = int(4.6e9 // per)
    g = torch.Generator().manual_seed(17)
    n = 3 * P
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(9, 16, D, generator=g).bfloat16().to(DEV)
    say(f"[gpu] past 4 GB {mode} pages={pages}")
    cache = fq.empty_kv_cache(pages, H, P, D, mode, DEV)
    where = [pages - 1, 0, pages - 2]
    slots = torch.cat([torch.arange(P) + p * P for p in where]).int().to(DEV)
    fq.kv_write(cache, k.to(DEV), v.to(DEV), slots)
    got = fq.attn_chunk(q, cache, _i32(*where)[None], _i32(0, 9), _i32(n))
    small, table = _one(k, v, mode, P)
    assert torch.equal(got, fq.attn_chunk(q, small, table, _i32(0, 9), _i32(n)))
