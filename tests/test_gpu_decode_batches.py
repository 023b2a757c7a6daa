"""GPU: attention of one new token in large batches (runs of more steps than a fetch of the block table covers, plans
over more sequences than a workgroup has threads), and the precision of its weights, against fp64."""
import math

import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, U, bound, softmax_attend, unpack, values
from gpu_util import DEV, say
from test_gpu_attention import _decode

MODES = ["bf16", "int8", "e4m3", "int4", "fp4"]


def _held(codes, scales, mode):
    """fp64 [pages, H, P, D] of a cache's side."""
    if mode in TDT:
        return codes.cpu().double()
    raw = unpack(codes.cpu().view(torch.uint8).numpy(), mode)
    return torch.from_numpy(values(raw, scales.cpu().numpy().astype(np.int64 if mode == "fp4" else np.float32), mode))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,H,D,per_cu", [("bf16", 8, 64, 4), ("bf16", 4, 128, 2), ("bf16", 2, 256, 1), ("int8", 8, 64, 4), ("int8", 4, 128, 2),
                                             ("int8", 4, 256, 2), ("e4m3", 4, 96, 2), ("e4m3", 8, 64, 4), ("int4", 6, 128, 3), ("int4", 8, 64, 4),
                                             ("fp4", 6, 128, 3), ("fp4", 4, 256, 2)])
def test_runs_longer_than_a_fetch_of_the_block_table(mode, H, D, per_cu):
    """Every workgroup's run holds more than 32 steps of 128 tokens, most from the middle of one sequence into the next.  The
    sequences share their pages, each in its own order; some miss a page far in, all end inside a tile."""
    B, P, most, g = 64, 64, 9000, 2
    pool = -(-most // P)
    rng, gen = np.random.default_rng(D + H), torch.Generator(device=DEV).manual_seed(D + H)
    cache = fq.empty_kv_cache(pool, H, P, D, mode, DEV)
    rows = lambda *s: torch.randn(s, generator=gen, device=DEV).bfloat16()  # noqa: E731
    fq.kv_write(cache, rows(pool * P, H, D), rows(pool * P, H, D), torch.arange(pool * P, dtype=torch.int32, device=DEV))
    table = np.stack([rng.permutation(pool) for _ in range(B)]).astype(np.int32)
    lens = most - rng.integers(0, 200, B)
    for b in range(0, B, 3):  # (tokens past 31 steps of the sequence, wherever a run begins)
        table[b, [70 + b % 9, 130]] = [-1, pool + 3]
    units = int(sum(-(-lens // 128))) * H
    assert units > 32 * 256 * per_cu
    say(f"[gpu] long runs {mode} H={H} D={D}: {units / (256 * per_cu):.0f} units a run")
    q = rows(B, g * H, D)
    lse = torch.empty(B, g * H, device=DEV)
    out = fq.attn_decode(q, cache, torch.from_numpy(table).to(DEV), torch.from_numpy(lens.astype(np.int32)).to(DEV), lse=lse).cpu().double()
    k, v = (_held(c, s, mode) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    q, lse = q.cpu().double(), lse.cpu().double()
    worst = 0.0
    for b in range(B):
        t = np.arange(lens[b])
        page = table[b, t // P]
        keep = (page >= 0) & (page < pool)
        page, off = page[keep], t[keep] % P
        n = len(page)
        want, wl, absv, top, vmax = softmax_attend(q[b:b + 1], k[page, :, off], v[page, :, off], torch.tensor([n]), 1 / math.sqrt(D))
        worst = max(worst, float(((out[b:b + 1] - want).abs() / bound(want, absv, top, vmax, n, D, "bf16", "bf16" if mode == "bf16" else "f16")).max()))
        assert ((lse[b:b + 1] - wl).abs() <= (D + 8) * 2.0 ** -24 * top + 2.0 ** -20 * (1 + wl.abs()) + math.sqrt(n) * 2.0 ** -23).all(), b
    say(f"[gpu]   worst error {worst:.3f} of its bound")
    assert worst <= 1.0


def _lengths(B, kind):
    """Mostly empty and short sequences with a few long ones, the longest at a place past 256 (and past 512)."""
    if kind == "empty":
        lens = [0] * B
    elif kind == "one":
        lens = [1] * B
    else:
        lens = [(7 * i * i + 3 * i) % 41 if i % 3 else 0 for i in range(B)]
    lens[B - 1] = 1500
    lens[min(B - 2, 300)] = 700
    if kind != "empty":
        lens[5] = 400
    return lens


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["empty", "one", "mixed"])
@pytest.mark.parametrize("B,mode,Hq,H,D", [(65, "int8", 4, 2, 64), (256, "same", 4, 2, 64), (257, "int8", 4, 2, 64), (512, "int4", 2, 1, 128), (513, "fp4", 12, 1, 64),
                                           (700, "e4m3", 2, 2, 64), (700, "same", 2, 1, 256), (1100, "int8", 3, 1, 32)])
def test_plans_over_many_sequences(B, mode, Hq, H, D, kind):
    """The run plan takes 256 sequences at a time and keeps the lengths of 512: batches on both sides of each, whose long
    sequences (split and joined) lie past them."""
    say(f"[gpu] batch {B} {kind} {mode} Hq={Hq} H={H} D={D}")
    _decode(_lengths(B, kind), Hq, H, D, 16, mode, "bf16", seed=B)


# ---- the weights' precision ---------------------------------------------------------------------------

# relative error of a weight: rounded once to 16 bits, or as the sum of two such roundings (the second of the first's
# remainder)
ONE, TWO = dict(U), {t: U[t] ** 2 for t in U}


def _pairs(B, Hq, D, n, seed):
    """Sequences whose tokens come in pairs of opposite values and nearly equal weights, so that outputs are far smaller than
    sum p |v| and their own rounding does not cover the weights'.  q, k small: scores within +-0.1 or so."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(B, Hq, D, generator=g), 0.05 * torch.randn(B, n, 1, D, generator=g)
    v = torch.randn(B, n // 2, 1, 1, generator=g).abs() + 0.5
    v = torch.stack([v, -v], 2).flatten(1, 2).expand(B, n, 1, D).contiguous()
    return q, k, v


def _weights_bound(out, absv, top, n, D, dt, u):
    """As attn_ref.bound, with u for a weight's rounding and nothing for weights far below the largest (there are none)."""
    rel = u + 2.0 * (D + 8) * 2.0 ** -24 * top[..., None] + (16 + math.sqrt(n)) * 2.0 ** -23
    return U[dt] * out.abs() + rel * absv * (1 + U[dt]) + 2.0 ** -25


def _pair_case(dt, mode, D=64, n=6, B=64, Hq=8):
    q, k, v = (t.to(TDT[dt]) for t in _pairs(B, Hq, D, n, 5))
    return q, k, v, (dt if mode in TDT else "f16")


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["same", "int8", "e4m3", "int4", "fp4"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Hq", [1, 3, 8])
def test_weights_count_in_two_parts(mode, dt, Hq):
    """With up to 8 heads on a cache head a weight's rounding to 16 bits is made good by its remainder."""
    mode = dt if mode == "same" else mode
    D, n, B, P = 64, 6, 64, 16
    q, k, v, p_dt = _pair_case(dt, mode, D, n, B, Hq)
    cache = fq.empty_kv_cache(B, 1, P, D, mode, DEV)
    slots = (torch.arange(B)[:, None] * P + torch.arange(n)).flatten().to(torch.int32).to(DEV)
    fq.kv_write(cache, k.flatten(0, 1).to(DEV), v.flatten(0, 1).to(DEV), slots)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    k64, v64 = (_held(c, s, mode)[:, :, :n].transpose(1, 2) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    for wide in (1, 80):  # (a workgroup a sequence; runs and their join)
        t = torch.cat([table, torch.full((B, wide), -1, dtype=torch.int32, device=DEV)], 1)
        out = fq.attn_decode(q.to(DEV), cache, t, lens).cpu().double()
        worst = 0.0
        for b in range(B):
            want, _, absv, top, _ = softmax_attend(q[b:b + 1].double(), k64[b], v64[b], torch.tensor([n]), 1 / math.sqrt(D))
            worst = max(worst, float(((out[b:b + 1] - want).abs() / _weights_bound(want, absv, top, n, D, dt, TWO[p_dt])).max()))
        say(f"[gpu] two parts {mode} {dt} Hq={Hq}: worst {worst:.3f} of its bound")
        assert worst <= 1.0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("mode", ["same", "int8"])
@pytest.mark.parametrize("Hq", [1, 3, 8])
def test_that_bound_tells_one_part_from_two(mode, dt, Hq):
    """(CPU) The same cases with the weights rounded once, everything else in fp64, are outside it; with two parts inside."""
    D, n, B = 64, 6, 64
    q, k, v, p_dt = _pair_case(dt, dt if mode == "same" else mode, D, n, B, Hq)
    worst = {1: 0.0, 2: 0.0}
    for b in range(B):
        k64, v64 = k[b].double(), v[b].double()
        want, _, absv, top, _ = softmax_attend(q[b:b + 1].double(), k64, v64, torch.tensor([n]), 1 / math.sqrt(D))
        s = (q[b].double() @ k64[:, 0].T) / math.sqrt(D)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        hi = p.to(TDT[p_dt]).double()
        lo = (p - hi).to(TDT[p_dt]).double()
        for parts, w in ((1, hi), (2, hi + lo)):
            o = ((w @ v64[:, 0]) / p.sum(-1, keepdim=True)).to(TDT[dt]).double()
            worst[parts] = max(worst[parts], float(((o - want[0]).abs() / _weights_bound(want, absv, top, n, D, dt, TWO[p_dt])[0]).max()))
    assert worst[1] > 1.5 and worst[2] < 1.0, worst
