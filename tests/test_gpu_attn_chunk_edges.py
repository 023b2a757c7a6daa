"""GPU: attention of new tokens over the paged cache where sums are not finite, scores large or values far from 1, in every row tile, in walks that one
workgroup has and in walks that are dealt in parts, against fp64 with the derived elementwise bound of attn_ref.bound."""
import math

import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, U, bound, encode, pack, values
from gpu_util import DEV, say
from test_gpu_attention import MODES, _check_rows
from test_gpu_attn_chunk import _i32, attend, seen_by

pytestmark = pytest.mark.gpu


def _cache(k, v, mode, dt, P=16):
    """A cache of one sequence with its pages in reverse, its table, and what it holds in fp64."""
    n, H, D = k.shape
    pages = -(-n // P)
    slots = (pages - 1 - torch.arange(n) // P) * P + torch.arange(n) % P
    m = dt if mode == "same" else mode
    cache = fq.empty_kv_cache(pages, H, P, D, m, "cpu")
    held = []
    for x, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        p, o = slots // P, slots % P
        if mode == "same":
            codes[p, :, o] = x
            held.append(x.double())
            continue
        code, sc = encode(x, mode)
        codes.view(torch.uint8)[p, :, o] = torch.from_numpy(pack(code, mode))
        scales[p, :, o] = torch.from_numpy(sc.astype("uint8") if mode == "fp4" else sc)
        held.append(torch.from_numpy(values(code, sc, mode)))
    dev = [None if t is None else t.to(DEV) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    return fq.KVCache(m, *dev), torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=DEV)[None], *held


# two query heads a cache head: row tiles of 32, 64 and 128
ROWS = [1, 20, 120]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [200, 2600])
@pytest.mark.parametrize("r", ROWS)
def test_infinities_in_16_bits(dt, D, n, r):
    """Infinities and NaN reach the rows that see them and no other, whatever part of a walk they lie in: one of a value stays an
    infinity however small its weight, two of other signs are NaN, a NaN key is a row's NaN."""
    say(f"[gpu] infinities {dt} D={D} keys={n} rows={r}")
    g = torch.Generator().manual_seed(30)
    H, G = 4, 2
    q, k, v = (torch.randn(m, h, D, generator=g).to(TDT[dt]) for m, h in ((r, H * G), (n, H), (n, H)))
    odd = []  # (key, cache head, element, value)
    for j, h, d, x in ((n // 3, 0, 7, math.inf), (n - r, 0, D - 1, -math.inf), (n - 1 - r // 2, 1, 9, math.nan), (n // 2, 2, 11, -math.inf),
                       (n // 5, 3, 33, math.inf), (n - 1 - r // 3, 3, 33, -math.inf)):
        v[j, h, d] = x
        odd.append((j, h, d))
    k[n // 2, 2] = -30.0 * q[r // 2, 2 * G]  # its weight is 0 in 32 bits for that row
    k[5, 0] = 2.0 * q[r // 2, 0]             # far from the infinities, a row's maximum
    k[n - 1 - r // 4, 1, 3] = math.nan
    for window, sinks in ((0, 0), (25, 3), (n - 30, 0)):
        cache, table, _, _ = _cache(k, v, "same", dt)
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), window, sinks).cpu().double()
        seen = seen_by(r, n, window, sinks)
        clean = [torch.where(torch.isfinite(t), t, 0.0).double() for t in (k, v)]
        out, _, absv, top, vmax = attend(q.double(), *clean, seen, 1 / math.sqrt(D))
        extra = torch.zeros(r, H * G, D, dtype=torch.float64)
        for j, h, d in odd:
            extra[seen[:, j], G * h:G * h + G, d] += float(v[j, h, d])
        extra[seen[:, n - 1 - r // 4], G:2 * G] = math.nan
        fin = extra == 0
        assert torch.equal(torch.isnan(got), torch.isnan(extra))
        assert torch.equal(got[~fin & ~extra.isnan()], extra[~fin & ~extra.isnan()])
        assert ((got - out).abs() <= bound(out, absv, top, vmax, n, D, dt, dt))[fin].all()


@pytest.mark.parametrize("mode", ["int8", "e4m3", "int4", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [200, 2600])
@pytest.mark.parametrize("r", ROWS)
def test_rows_that_are_not_finite_in_low_bits(mode, D, n, r):
    """A cached row (E2M1: a group) that reads back as NaN makes NaN of the rows that see it, and only of those."""
    say(f"[gpu] not finite {mode} D={D} keys={n} rows={r}")
    g = torch.Generator().manual_seed(31)
    H, G = 4, 2
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, H * G), (n, H), (n, H)))
    k[n - 1 - r // 4, 1, 3], v[n // 3, 0, 40], v[n - 1 - r // 2, 2, 1] = math.nan, math.inf, math.nan
    second, first = (slice(32, 64), slice(32)) if mode == "fp4" else (slice(D), slice(D))  # what the values' NaN and infinity reach of a row
    cache, table, _, _ = _cache(k, v, mode, "bf16")
    clean = _cache(torch.where(torch.isfinite(k), k, 0.0), torch.where(torch.isfinite(v), v, 0.0), mode, "bf16")
    kk, vv = clean[2:]
    vv[n // 3, 0, second], vv[n - 1 - r // 2, 2, first] = 0.0, 0.0
    for window, sinks in ((0, 0), (25, 3), (n - 30, 0)):
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), window, sinks).cpu().double()
        seen = seen_by(r, n, window, sinks)
        bad = torch.zeros(r, H * G, D, dtype=torch.bool)
        bad[seen[:, n - 1 - r // 4], G:2 * G] = True
        bad[seen[:, n // 3], :G, second] = True
        bad[seen[:, n - 1 - r // 2], 2 * G:3 * G, first] = True
        assert torch.equal(torch.isnan(got), bad)
        out, _, absv, top, vmax = attend(q.double(), kk, vv, seen, 1 / math.sqrt(D))
        assert ((got - out).abs() <= bound(out, absv, top, vmax, n, D, "bf16", "f16"))[~bad].all()


@pytest.mark.parametrize("mode", ["int8", "e4m3", "int4", "fp4"])
@pytest.mark.parametrize("e", [90, 104, 112, 118, 125])
def test_many_small_weights_beside_large_values(mode, e):
    """4000 keys 9 to 12 nats below the one that stands out hold a third of the weight: with values of any size (2^e and its neighbours)
    they count, in the result and in lse."""
    n, D, G = 4000, 64, 8
    g = torch.Generator().manual_seed(32)
    for r in (1, 6, 16):
        say(f"[gpu] small weights {mode} e={e} rows={r}")
        q = torch.zeros(r, G, D, dtype=torch.bfloat16)
        q[..., 0] = 8.0
        k = torch.zeros(n, 1, D)
        k[:, 0, 0] = -(torch.rand(n, generator=g) * 3 + 9)
        k[7] = 0.0
        k[n - r:, 0, 0] = -30.0
        v = ((0.5 + torch.rand(n, 1, D, generator=g)) * 2.0 ** e).bfloat16()
        cache, table, kk, vv = _cache(k.bfloat16(), v, mode, "bf16")
        lse = torch.empty(r, G, device=DEV)
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), lse=lse).cpu()
        want = attend(q.double(), kk, vv, seen_by(r, n, 0, 0), 1 / math.sqrt(D))
        assert want[1].min() > 0.1
        _check_rows(got, lse.cpu(), want, "bf16", D, n, "f16", f"{mode} 2^{e}")


@pytest.mark.parametrize("mode", ["int8", "e4m3", "int4", "fp4"])
@pytest.mark.parametrize("e", [60, 100, 125])
def test_rows_before_large_values(mode, e):
    """Rows that see a token's values of 2^e and, in the same tile, rows that do not and whose own are ordinary: all within the bound."""
    n, D, G, H = 1900, 64, 2, 2
    for r in (6, 20, 120):
        say(f"[gpu] before large values {mode} e={e} rows={r}")
        g = torch.Generator().manual_seed(34)
        q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, H * G), (n, H), (n, H)))
        v[n - 1 - r // 3] *= 2.0 ** e
        cache, table, kk, vv = _cache(k, v, mode, "bf16")
        lse = torch.empty(r, H * G, device=DEV)
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), lse=lse).cpu()
        # (rows in two groups: the bound's largest value is one that a row sees)
        before = r - 1 - r // 3
        for rows, m in ((slice(before), n - r + before), (slice(before, r), n)):
            *want, top = attend(q[rows].double(), kk[:m], vv[:m], seen_by(r, n, 0, 0)[rows, :m], 1 / math.sqrt(D))
            # A weight times its value's scale is held to 2^-30 of the row's largest of these, for all elements alike: that times a code is
            # up to 2^-30 of the largest value of any element (127, 448, 7 or 6 times its scale), also where the large token's own code is 0.
            _check_rows(got[rows], lse.cpu()[rows], (*want, top.amax(-1, keepdim=True).expand_as(top)), "bf16", D, m, "f16", f"{mode} rows {rows}")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1e3, 1e7, -1e9, 1e15, 1e30])
def test_scores_of_any_size(mode, dt, scale):
    """Scores far past what fp32 tells apart by less than 1 still give means of the values that are seen, and the value of the
    key that stands out where one does by more than the scores' own error, (D + 8) 2^-24 of their terms."""
    n, D, G = 2100, 64, 4
    for r in (1, 12, 40):
        say(f"[gpu] scores {mode} {dt} scale={scale} rows={r}")
        g = torch.Generator().manual_seed(33)
        q, k, v = (torch.randn(m, h, D, generator=g).to(TDT[dt]) for m, h in ((r, G), (n, 1), (n, 1)))
        cache, table, kk, vv = _cache(k, v, mode, dt)
        got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n), scale=scale).cpu().double()
        seen = seen_by(r, n, 0, 0)
        s = (torch.einsum("ihd,jd->ihj", q.double(), kk[:, 0]) * scale).masked_fill(~seen[:, None], -math.inf)
        off = torch.einsum("ihd,jd->ihj", q.double().abs(), kk[:, 0].abs()).amax(-1) * abs(scale) * (D + 8) * 2.0 ** -24
        top = s.topk(2, -1)
        u = U[dt]
        least, most = vv[:, 0].amin(0), vv[:, 0].amax(0)
        assert torch.isfinite(got).all()
        assert (got >= least - 3 * u * least.abs()).all() and (got <= most + 3 * u * most.abs()).all()
        clear = top.values[..., 0] - top.values[..., 1] > 2 * off + 60
        assert clear.any()
        one = vv[:, 0][top.indices[..., 0]]
        assert ((got - one).abs() <= 3 * u * one.abs() + 2.0 ** -24)[clear].all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("r", [1, 4, 8])
def test_weights_of_few_rows_keep_their_bits(mode, dt, r):
    """Two kinds of keys whose values cancel, so that what a weight's rounding adds shows in the output: with weights in two parts it is 2^-16 of
    sum p |v| for bf16 operands and 2^-22 for f16 ones, as fq_attn_decode's.  Tiles of 32 rows, and of 64 where the rows' type has
    the weights' bits."""
    n, D, G, H = 1000, 64, 8, 1
    if r * G > 32 and mode != "same" and dt == "bf16":
        return
    say(f"[gpu] weights {mode} {dt} rows={r}")
    g = torch.Generator().manual_seed(35)
    q = torch.zeros(r, G, D)
    q[..., 0] = 0.25 * torch.arange(1, G + 1)  # (other weights for each head)
    k, v = torch.zeros(n, H, D), torch.ones(n, H, D)
    k[::2, :, 0], v[::2] = -2.0, -1.3
    q, k, v = q.to(TDT[dt]), k.to(TDT[dt]), (v * (1 + 0.2 * torch.rand(1, 1, D, generator=g))).to(TDT[dt])
    cache, table, kk, vv = _cache(k, v, mode, dt)
    got = fq.attn_chunk(q.to(DEV), cache, table, _i32(0, r), _i32(n)).cpu().double()
    out, _, absv, top, _ = attend(q.double(), kk, vv, seen_by(r, n, 0, 0), 1 / math.sqrt(D))
    # attn_ref.bound with these weights: scores, exp and sums as there
    rel = (2.0 ** -16 if mode == "same" and dt == "bf16" else 2.0 ** -22) + (2.0 ** -17 if mode != "same" else 0.0)
    rel = rel + 2.0 * (D + 8) * 2.0 ** -24 * top[..., None] + (16 + math.sqrt(n)) * 2.0 ** -23
    assert (out.abs() < 0.1 * absv).any()
    tol = U[dt] * out.abs() + rel * absv * (1 + U[dt]) + n * 2.0 ** -40 * vv.abs().max() + (2.0 ** -25 if dt == "f16" else 0.0)
    worst = ((got - out).abs() / tol).max().item()
    say(f"[gpu]   worst error {worst:.3f} of its bound")
    assert worst <= 1


def test_row_numbers_far_below_zero():
    """A cu_q that does not ascend, down to the smallest int32: a sequence has no rows then (a difference of these numbers passes 32 bits), and
    those of the sequences beside it are right."""
    g = torch.Generator().manual_seed(36)
    r, n, D = 40, 300, 64
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, 4), (n, 2), (n, 2)))
    cache, table, kk, vv = _cache(k, v, "same", "bf16")
    want, _, absv, top, vmax = attend(q.double(), kk, vv, seen_by(r, n, 0, 0), 1 / math.sqrt(D))
    tol = bound(want, absv, top, vmax, n, D, "bf16", "bf16")
    for low in (-1, -2 ** 31, -2 ** 31 + 39):
        for cu in ((0, r, low, low), (r, low, r)):
            say(f"[gpu] cu_q {cu}")
            out = torch.full((r, 4, D), 7.0, dtype=torch.bfloat16, device=DEV)
            B = len(cu) - 1
            fq.attn_chunk(q.to(DEV), cache, table.expand(B, -1), _i32(*cu), _i32(*[n] * B), out=out)
            assert ((out.cpu().double() - want).abs() <= tol).all()
