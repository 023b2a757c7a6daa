"""GPU: attention at the edges of its inputs' ranges, against fp64 or known results."""
import math

import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import bound, softmax_attend
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
TDT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _cached(k, v, mode, P=16):
    """A cache of one sequence and its table."""
    n, H, D = k.shape
    pages = -(-n // P)
    cache = fq.empty_kv_cache(pages, H, P, D, mode, DEV)
    fq.kv_write(cache, k, v, torch.arange(n, dtype=torch.int32, device=DEV))
    return cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None]


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("scale", [1e-50, -1e-50, 1e-300, 1e-45, 3e-39])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_scales_below_fp32(scale, dt):
    """Every weight is 1 (to far below a rounding): row i gives the mean of the values it sees."""
    g = torch.Generator().manual_seed(1)
    n, Hq, H, D = 200, 4, 2, 64
    q, k, v = (torch.randn(n, h, D, generator=g).to(TDT[dt]) for h in (Hq, H, H))
    mean = (v.double().cumsum(0) / torch.arange(1, n + 1)[:, None, None]).repeat_interleave(Hq // H, 1)
    # the output's rounding, the sums' 200 terms in fp32, and a bf16 (f16) rounding of weights that are exactly 1: none
    tol = 2.0 ** (-8 if dt == "bf16" else -11) * mean.abs() + 200 * 2.0 ** -24 * 4.0 + 2.0 ** -25
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    lse = torch.empty(n, Hq, device=DEV)
    say(f"[gpu] scale {scale} {dt}")
    got = fq.attn_prefill(q, k, v, _i32(0, n), scale=scale, lse=lse).cpu().double()
    assert ((got - mean).abs() <= tol).all()
    want = torch.log(torch.arange(1, n + 1, dtype=torch.float64))[:, None]
    assert ((lse.cpu().double() - want).abs() <= 2.0 ** -20).all()
    cache, table = _cached(k, v, dt)
    got = fq.attn_decode(q[-1:], cache, table, _i32(n), scale).cpu().double()
    assert ((got[0] - mean[-1]).abs() <= tol[-1]).all()


@pytest.mark.parametrize("mode", ["bf16", "int8", "e4m3", "int4", "fp4"])
def test_the_largest_scales(mode):
    """A scale of 2^127 with one key that is not zero: scores of 0 and one of +-2^127 or so, no NaN."""
    n, H, D = 40, 1, 64
    q = torch.zeros(1, H, D)
    q[0, 0, 5] = 1.0
    k = torch.zeros(n, H, D)
    v = torch.arange(1, n + 1).float()[:, None, None].expand(n, H, D).contiguous()
    for sign in (1.0, -1.0):
        k[7, 0, 5] = sign
        qd, kd, vd = q.bfloat16().to(DEV), k.bfloat16().to(DEV), v.bfloat16().to(DEV)
        cache, table = _cached(kd, vd, mode)
        kept = fq.kv_read(cache, table, _i32(0, n), n, torch.bfloat16)[1].cpu().double()
        seen = kept[7, 0] if sign > 0 else torch.cat([kept[:7], kept[8:]])[:, 0].mean(0)
        for scale in (2.0 ** 127, 2.0 ** 120):
            got = [fq.attn_decode(qd, cache, table, _i32(n), scale)]
            if mode == "bf16":
                got.append(fq.attn_prefill(qd, kd, vd, _i32(0, 1), _i32(0, n), scale=scale))
            for o in got:  # (the output's rounding to bf16, and 40 terms' in fp32)
                assert ((o[0, 0].cpu().double() - seen).abs() <= seen.abs() * (2.0 ** -8 + 2.0 ** -18)).all()


def _one_low_key(n, H, Hq, D, dt, at, nats, sign, seed):
    """Keys whose scores are 0 but that of token `at`, `nats` below; its value's element 3 of head 0 is infinite."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.ones(1, Hq, D), torch.zeros(n, H, D)
    k[at] = -nats / math.sqrt(D)
    v = torch.randn(n, H, D, generator=g)
    v[at, 0, 3] = sign * math.inf
    return (t.to(TDT[dt]).to(DEV) for t in (q, k, v))


def _check_infinity(o, v, at, Hq, H, sign, dt, label):
    """Element 3 of head 0's group is infinite, everything else the mean of the other tokens' values (the low one's weight is
    below their rounding: e^-12 / 40 = 1.5e-7)."""
    rest = torch.cat([v[:at], v[at + 1:]]).double().cpu()
    mean = rest.mean(0).repeat_interleave(Hq // H, 0)
    o = o.double().cpu()
    hit = torch.zeros(o.shape, dtype=torch.bool)
    hit[: Hq // H, 3] = True
    assert (o[hit] == sign * math.inf).all(), (label, o[hit])
    tol = 2.0 ** (-8 if dt == "bf16" else -11) * mean.abs() + 2.0 ** -17 * 4.0
    assert ((o - mean).abs() <= tol)[~hit].all(), label


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,H,D", [(2, 2, 64), (8, 1, 128), (8, 2, 96), (12, 1, 64), (20, 1, 256), (4, 1, 256), (40, 2, 128)])
def test_an_infinity_with_a_small_weight_stays_one(dt, Hq, H, D):
    """However small the weight of the token that holds it (one that f16, and one that fp32, has no number for), wherever it
    lies: before the maximum moves, after it, in a part of its own."""
    for n, P in ((40, 16), (300, 32), (2100, 16)):
        for at in (0, n // 2, n - 1):
            for nats in (12.0, 17.5, 40.0, 100.0, 400.0):
                sign = 1.0 if at else -1.0
                label = f"decode {dt} Hq={Hq} H={H} D={D} n={n} at={at} nats={nats}"
                q, k, v = _one_low_key(n, H, Hq, D, dt, at, nats, sign, n + at)
                cache, table = _cached(k, v, dt, P)
                wide = torch.cat([table, torch.full((1, 40), -1, dtype=torch.int32, device=DEV)], 1)
                for t in (table, wide):  # (a workgroup a segment where the table is short; split and joined)
                    _check_infinity(fq.attn_decode(q, cache, t, _i32(n))[0], v, at, Hq, H, sign, dt, label)
    say(f"[gpu] {label}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,H,D", [(2, 2, 64), (8, 1, 128), (4, 1, 96), (3, 1, 256)])
def test_a_prompts_infinity_with_a_small_weight_stays_one(dt, Hq, H, D):
    """In whole and in partly masked tiles, and in walks cut into parts; rows before the token do not see it."""
    for n, rows in ((300, 300), (300, 3), (4000, 1), (4000, 40)):
        for at in (5, n // 2, n - 2):
            for nats in (12.0, 17.5, 40.0, 100.0, 400.0):
                label = f"prompt {dt} Hq={Hq} H={H} D={D} {rows} behind {n} at={at} nats={nats}"
                q, k, v = _one_low_key(n, H, Hq, D, dt, at, nats, 1.0, n + at)
                q = q.repeat(rows, 1, 1)
                o = fq.attn_prefill(q, k, v, _i32(0, rows), _i32(0, n))
                assert not o.isnan().any(), label
                first = max(0, at - (n - rows))  # the first row that sees the token
                assert not o[:first].isinf().any() and (o[first:, : Hq // H, 3] == math.inf).all(), label
                assert o.isinf().sum() == (rows - first) * (Hq // H), label
                _check_infinity(o[-1], v, at, Hq, H, 1.0, dt, label)
                full = fq.attn_prefill(q, k, v, _i32(0, rows), _i32(0, n), causal=False)
                _check_infinity(full[0], v, at, Hq, H, 1.0, dt, label)
    say(f"[gpu] {label}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_infinities_of_both_signs_give_nan(dt):
    n, Hq, H, D = 700, 8, 1, 64
    q, k, v = _one_low_key(n, H, Hq, D, dt, 20, 30.0, 1.0, 1)
    v[650, 0, 3], v[4, 0, 9], v[40, 0, 60] = -math.inf, math.nan, -math.inf
    cache, table = _cached(k, v, dt)
    for o in (fq.attn_decode(q, cache, table, _i32(n)), fq.attn_prefill(q, k, v, _i32(0, 1), _i32(0, n))):
        odd = o[0].isnan()
        assert odd[:, [3, 9]].all() and odd.sum() == 2 * Hq and (o[0, :, 60] == -math.inf).all() and o.isinf().sum() == Hq


# ---- many tokens far below one that stands out ------------------------------------------------------

def _sink(n, H, Hq, D, dt, at, nats, seed):
    """Token `at` scores `nats` above all others, which score 0, and has a value of 0; the others' values are near 1."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.ones(1, Hq, D), torch.zeros(n, H, D)
    k[at] = nats / math.sqrt(D)
    v = 1.0 + 0.25 * torch.rand(n, H, D, generator=g)
    v[at] = 0.0
    return (t.to(TDT[dt]).to(DEV) for t in (q, k, v))


def _sink_want(k, v, D):
    """fp64: out [H, D] of the rows as they are kept (q all ones), and the largest |v|."""
    s = k.double().cpu().sum(-1) / math.sqrt(D)
    p = torch.softmax(s, 0)
    return (p[..., None] * v.double().cpu()).sum(0), float(v.double().abs().max())


def _sink_check(o, want, vmax, n, dt, p_bits, g, label):
    """The output's rounding, 2^-11 (2^-8 in bf16) of it; the weights': 2^-11 relative (2^-8 where bf16 products take them
    once) or `p_bits` bits below the largest, whichever is more; scores of 17 in fp32 to 2^-20, sums of n terms."""
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    tol = want.abs() * (2 * u + 2.0 ** -18 + math.sqrt(n) * 2.0 ** -23) + n * 2.0 ** -p_bits * vmax + 2.0 ** -25
    o = o.double().cpu()
    want, tol = (t.repeat_interleave(g, 0) for t in (want, tol))
    worst = float(((o - want).abs() / tol).max())
    say(f"[gpu] {label}: worst {worst:.3f} of its bound")
    assert worst <= 1.0, label


@pytest.mark.parametrize("mode", ["f16", "bf16", "int8", "e4m3", "int4", "fp4"])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 64), (16, 1, 128), (12, 1, 256), (9, 1, 96)])
def test_many_tokens_far_below_one(mode, Hq, H, D):
    """20000 tokens, each with 2.5e-8 of the largest weight, make 5e-4 of the sum: below f16's smallest number one by one.
    Weights are held to 2^-32 of the largest (2^-30 with a scale a token) and in two parts with up to 8 heads a group.  Alone
    the sequence is cut into many runs, most without the large weight; 520 times (in the same pages) into few."""
    n, nats = 20000, 17.5
    for dt in ("f16", "bf16") if mode not in ("f16", "bf16") else (mode,):
        for at in (0, 10007):
            q, k, v = _sink(n, H, Hq, D, dt, at, nats, 3)
            cache, table = _cached(k, v, mode, 64)
            kk, vv = (k, v) if mode == dt else fq.kv_read(cache, table, _i32(0, n), n, torch.float16)
            want, vmax = _sink_want(kk, vv, D)
            bits = 35 if Hq <= 8 else 32 if mode in ("f16", "bf16", "fp4") else 30
            for B in (1, 520):
                o = fq.attn_decode(q.repeat(B, 1, 1), cache, table.repeat(B, 1), _i32(n).repeat(B))
                for b in {0, B // 2, B - 1}:
                    _sink_check(o[b], want, vmax, n, dt, bits, Hq // H, f"{mode} {dt} Hq={Hq} D={D} at={at} {b} of {B}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,H,D", [(2, 1, 64), (2, 2, 128), (1, 1, 200)])
def test_a_prompts_many_tokens_far_below_one(dt, Hq, H, D):
    n, nats = 20000, 17.5
    for at in (0, 10007):
        q, k, v = _sink(n, H, Hq, D, dt, at, nats, 4)
        want, vmax = _sink_want(k, v, D)
        for rows in (1, 200):
            o = fq.attn_prefill(q.repeat(rows, 1, 1), k, v, _i32(0, rows), _i32(0, n))
            _sink_check(o[-1], want, vmax, n, dt, 32, Hq // H, f"prompt {dt} Hq={Hq} D={D} at={at} rows={rows}")


@pytest.mark.parametrize("Hq,H,D", [(4, 1, 64), (16, 1, 128), (2, 1, 256), (6, 2, 96)])
def test_e2m1_groups_of_very_different_sizes(Hq, H, D):
    """A group of 32 far smaller than its tokens' others counts with all its bits where it is what matters: keys 2^26 smaller,
    under a q that is 0 for the others; values 2^25 smaller, whose outputs are their own."""
    n = 200
    g = torch.Generator().manual_seed(6)
    code = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])[torch.randint(0, 8, (2, n, H, D), generator=g)]
    code *= torch.where(torch.rand(code.shape, generator=g) < 0.5, -1.0, 1.0)
    code[..., ::32] = 6.0  # (the group's largest: its exponent is then the size's)
    size = torch.ones(2, D)
    size[0, 32:64], size[1, 32:64] = 2.0 ** -26, 2.0 ** -25
    k, v = (code[i] * size[i] for i in range(2))
    q = torch.zeros(1, Hq, D)
    q[..., 32:64] = 2.0 ** 24 * torch.randn(1, Hq, 32, generator=g)
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    cache, table = _cached(k.to(DEV), v.to(DEV), "fp4")
    kept = fq.kv_read(cache, table, _i32(0, n), n, torch.bfloat16)
    assert torch.equal(kept[0].cpu(), k) and torch.equal(kept[1].cpu(), v)
    out, _, absv, top, vmax = softmax_attend(q.double(), k.double(), v.double(), torch.tensor([n]), 1 / math.sqrt(D))
    o = fq.attn_decode(q.to(DEV), cache, table, _i32(n)).cpu().double()
    worst = ((o - out).abs() / bound(out, absv, top, vmax, n, D, "bf16", "f16")).max()
    say(f"[gpu] groups Hq={Hq} H={H} D={D}: worst {float(worst):.3f} of its bound")
    assert worst <= 1.0
