"""GPU: norms and rotation of queries and keys, and the cache append, against the formulas in fp64."""
import math

import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import E2M1, TDT, U, unpack, values
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
EPS = 1e-6
MODES = ["same", "int8", "e4m3", "int4", "fp4"]


def turned(x, weight, positions, inv_freq, axes, interleaved, eps=EPS):
    """(result, bound of the fp32 result's error) of rows x [T, heads, D], all fp64 on the host.  The bound: the norm's
    factor is off by its sum (at most D / 8 + 8 additions one after the other, halved by the root), mean, root, quotient
    and two products: (D / 16 + 12) 2^-24.  Sine and cosine are off by their argument's rounding to fp32 (half turns of at
    most 1: pi 2^-25), the function's 2 ulp and the fp64 phase (two roundings of it): 3 2^-23 + 4 pi |turns| 2^-53.  Two products and
    a sum: 3 2^-24."""
    x = x.double()
    T, _, D = x.shape
    rel = 0.0
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
        rel = (D / 16 + 12) * 2.0 ** -24
    half = inv_freq.numel()
    R = 2 * half
    pos = positions.double().reshape(-1, T)
    which = torch.zeros(half, dtype=torch.long) if axes is None else axes.long()
    ok = (which >= 0) & (which < pos.shape[0])
    p = torch.where(ok[None], pos.T[:, which.clamp(0, pos.shape[0] - 1)], 0.0)  # [T, half]
    turns = p * inv_freq.double() / (2 * math.pi)
    t = (2 * math.pi * (turns - turns.round()))[:, None]
    ang = (3 * 2.0 ** -23 + 4 * math.pi * turns.abs() * 2.0 ** -53)[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :half], x[..., half:R])
    u, v = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    e = (a.abs() + b.abs()) * (rel + ang + 3 * 2.0 ** -24)
    join = lambda m, n: torch.stack([m, n], -1).flatten(-2) if interleaved else torch.cat([m, n], -1)  # noqa: E731
    return torch.cat([join(u, v), x[..., R:]], -1), torch.cat([join(e, e), x[..., R:].abs() * rel], -1)


def rounded(want, err, dt):
    """Bound of the error once rounded to dt (f16's subnormals are 2^-24 apart)."""
    return err + U[dt] * (want.abs() + err) + (2.0 ** -25 if dt == "f16" else 0.0)


def freqs(R, base=1e4):
    return (base ** (-torch.arange(R // 2, dtype=torch.float64) / max(1, R // 2))).float()


def make(T, Hq, Hkv, D, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g) * torch.exp(torch.empty(T, Hq + 2 * Hkv, 1).uniform_(-spread, spread, generator=g))
    return x.to(TDT[dt]), g


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# T, Hq, Hkv, D, R
SIZES = [(1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (3, 5, 2, 64, 32), (7, 16, 16, 80, 80), (33, 4, 4, 256, 256), (130, 7, 1, 96, 40), (5, 3, 1, 72, 72),
         (2000, 8, 2, 128, 64), (65, 2, 1, 40, 24), (9, 12, 3, 160, 0), (4, 2, 2, 136, 136)]


@pytest.mark.parametrize("T,Hq,Hkv,D,R", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, "f32", "own", "one"])
def test_rope(T, Hq, Hkv, D, R, dt, interleaved, norm):
    say(f"[gpu] rope {dt} T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} interleaved={interleaved} norm={norm}")
    x, g = make(T, Hq, Hkv, D, dt, T * D + R)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    wq = None if norm is None else (1 + 0.3 * torch.randn(D, generator=g)).to(torch.float32 if norm == "f32" else TDT[dt])
    wk = None if norm in (None, "one") else (1 + 0.3 * torch.randn(D, generator=g)).to(wq.dtype)
    pos = torch.randint(-5000, 100000, (T,), generator=g, dtype=torch.int32)
    f = freqs(R)
    xd = x.to(DEV)
    qd, kd = xd[:, :Hq], xd[:, Hq:Hq + Hkv]  # strided views
    got = fq.qk_rope(qd, kd, *dev(pos, f), *dev(wq, wk), EPS, interleaved)
    for o, src, w in zip(got, (q, k), (wq, wk)):
        want, err = turned(src, w, pos, f, None, interleaved)
        assert o.shape == src.shape and o.is_contiguous()
        off = (o.cpu().double() - want).abs() - rounded(want, err, dt)
        assert (off <= 0).all(), (off.max().item(), np.unravel_index(off.argmax().item(), off.shape))
    assert torch.equal(xd.cpu(), x)
    # one side alone, and into the input itself: the same bits
    q1, none = fq.qk_rope(qd, None, *dev(pos, f), *dev(wq, None), EPS, interleaved)
    none2, k1 = fq.qk_rope(None, kd, *dev(pos, f), *dev(None, wk), EPS, interleaved)
    assert none is None and none2 is None and torch.equal(q1, got[0]) and torch.equal(k1, got[1])
    fq.qk_rope(qd, kd, *dev(pos, f), *dev(wq, wk), EPS, interleaved, q_out=qd, k_out=kd)
    assert torch.equal(qd, got[0]) and torch.equal(kd, got[1]) and torch.equal(xd[:, Hq + Hkv:].cpu(), x[:, Hq + Hkv:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("A", [1, 2, 3, 16])
def test_axes(A, interleaved):
    T, H, D, R = 37, 3, 128, 96
    x, g = make(T, H, 0, D, "bf16", A)
    pos = torch.randint(0, 3000, (A, T + 5), generator=g, dtype=torch.int32)[:, :T]
    axes = torch.randint(0, A, (R // 2,), generator=g, dtype=torch.int32)
    axes[3], axes[-1] = A, -1  # no axis: not turned
    f = freqs(R)
    pd = torch.zeros(A, T + 5, dtype=torch.int32, device=DEV)
    pd[:, :T] = pos.to(DEV)
    got, _ = fq.qk_rope(x.to(DEV), None, pd[:, :T], f.to(DEV), interleaved=interleaved, axes=axes.to(DEV))
    want, err = turned(x, None, pos, f, axes, interleaved)
    assert ((got.cpu().double() - want).abs() <= rounded(want, err, "bf16")).all()
    if A == 1:  # one axis for all is the plain form
        one = torch.zeros(R // 2, dtype=torch.int32, device=DEV)
        a, _ = fq.qk_rope(x.to(DEV), None, pd[:, :T], f.to(DEV), interleaved=interleaved, axes=one)
        b, _ = fq.qk_rope(x.to(DEV), None, pd[0, :T], f.to(DEV), interleaved=interleaved)
        assert torch.equal(a, b)


def test_far_positions():
    """Angles keep their accuracy up to the ends of the positions' type."""
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x, _ = make(len(pos), 2, 0, 64, "f16", 5)
    f = freqs(64)
    got, _ = fq.qk_rope(x.to(DEV), None, *dev(pos, f))
    want, err = turned(x, None, pos, f, None, False)
    assert ((got.cpu().double() - want).abs() <= rounded(want, err, "f16")).all()
    assert torch.equal(got[0].cpu(), x[0])  # position 0 changes nothing


def test_infinities_stay_in_their_rows():
    x, g = make(6, 3, 1, 64, "bf16", 7)
    x[1, 0, 5], x[3, 1, 63], x[4, 3, 40] = math.inf, math.nan, -math.inf
    w = torch.ones(64)
    f, pos = freqs(32), torch.arange(6, dtype=torch.int32)
    for weight in (None, w):
        got = torch.cat(fq.qk_rope(*dev(x[:, :3].contiguous(), x[:, 3:4].contiguous(), pos, f, weight, weight)), 1).cpu()
        clean = torch.isfinite(x[:, :4]).all(-1)
        assert clean.sum() == 6 * 4 - 3 and torch.isfinite(got[clean]).all()
        want, err = turned(x[:, :4], weight, pos, f, None, False)
        assert ((got.double() - want).abs() <= rounded(want, err, "bf16"))[clean].all()
        # an element past the turned ones and without a norm touches only itself
        if weight is None:
            assert torch.isnan(got[3, 1, 63]) and torch.isfinite(got[3, 1, :63]).all()


def _held_ok(raw, scale, want, err, mode, clip, dmax):
    """Codes and scales of rows whose exact values are `want` [n, D] to within `err`."""
    code = unpack(raw, mode)
    scale = scale.astype(np.int64) if mode == "fp4" else scale
    got = values(code, scale, mode)
    D = want.shape[-1]
    if mode == "fp4":
        top, e = (np.abs(t).reshape(*t.shape[:-1], D // 32, 32).max(-1) for t in (want, err))
        g8 = scale[..., :D // 32]

        def e8_of(t):
            if dmax == 0.0:
                return np.where(t > 0, np.floor(np.log2(np.maximum(t, 1e-300))), -200) - 2 + 127
            return np.where(t > 0, np.ceil(np.log2(np.maximum(t, 1e-300) / dmax)), -200) + 127
        lo, hi = e8_of((top - e) * (1 - 2.0 ** -22)), e8_of((top + e) * (1 + 2.0 ** -22))
        assert ((g8 >= np.clip(lo, 0, 254)) & (g8 <= np.clip(hi, 0, 254))).all()
        unit = np.repeat(np.ldexp(1.0, (g8 - 127).astype(int)), 32, -1)
        y = np.abs(want) / unit
        half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0)) * unit  # half of E2M1's step
        room = np.where(y > 6, np.abs(want) - 6 * unit, 0.0)              # saturated
        assert (np.abs(got - want) <= half + room + 2 * err).all()
        return
    top, e = np.abs(want).max(-1), np.abs(err).max(-1)
    qmax = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}[mode] / clip
    assert (np.abs(scale - top / qmax) <= e / qmax + top / qmax * 2.0 ** -22).all()
    s = scale[..., None].astype(np.float64)
    half = 0.5 * s if mode != "e4m3" else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)
    cap = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}[mode] * s
    room = np.maximum(np.abs(want) - cap, 0.0)
    assert (np.abs(got - want) <= half * (1 + 2.0 ** -20) + room + 2 * err).all()


def _gathered(cache, slots):
    P = cache.page_size
    pick = lambda t: None if t is None else t.contiguous().cpu().view(torch.uint8 if t.dtype != torch.float32 else torch.float32).numpy()  # noqa: E731
    out = []
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c, s = pick(c), pick(s)
        out.append((np.stack([c[i // P, :, i % P] for i in slots]), None if s is None else np.stack([s[i // P, :, i % P] for i in slots])))
    return out


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,P,norm,interleaved,clip,dmax",
                         [(1, 4, 1, 64, 64, 16, True, False, 1.0, 0.0), (45, 8, 2, 128, 128, 16, True, False, 1.0, 0.0),
                          (70, 0, 3, 96, 48, 64, False, True, 0.9, 7.0), (600, 6, 6, 256, 256, 32, True, False, 1.0, 8.0),
                          (33, 8, 8, 160, 160, 16, False, False, 1.0, 0.0)])
def test_append(mode, dt, T, Hq, Hkv, D, R, P, norm, interleaved, clip, dmax):
    m = dt if mode == "same" else mode
    say(f"[gpu] append {m} {dt} T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} P={P}")
    x, g = make(T, Hq, Hkv, D, dt, 11 * T + D, 4.0)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(TDT[dt]) if norm else None for _ in range(2))
    pos, f = torch.randint(0, 70000, (T,), generator=g, dtype=torch.int32), freqs(R)
    pages = -(-T // P) + 2
    slots = np.random.default_rng(T).permutation(pages * P)[:T].astype(np.int32)
    gone = np.zeros(T, bool)
    if T > 8:
        gone[[2, 5]] = True
    where = slots.copy()
    where[gone] = [-3, pages * P + 1][:gone.sum()]
    cache, plain = (fq.empty_kv_cache(pages, Hkv, P, D, m, DEV) for _ in range(2))
    for c in (cache, plain):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0x55)
    xd = x.to(DEV)
    out = fq.kv_append(cache, xd[:, :Hq] if Hq else None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], torch.from_numpy(where).to(DEV), *dev(pos, f, wq if Hq else None, wk),
                       EPS, interleaved, None, clip, dmax)
    if Hq:
        only, _ = fq.qk_rope(xd[:, :Hq], None, *dev(pos, f, wq), None, EPS, interleaved)
        assert torch.equal(out, only)
        want, err = turned(q, wq, pos, f, None, interleaved)
        assert ((out.cpu().double() - want).abs() <= rounded(want, err, dt)).all()
    # the values, and what no slot names, are what the cache's own write leaves
    fq.kv_write(plain, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], torch.from_numpy(where).to(DEV), clip, dmax)
    (gk, gks), (gv, gvs) = _gathered(cache, np.arange(pages * P))
    (pk, pks), (pv, pvs) = _gathered(plain, np.arange(pages * P))
    assert (gv == pv).all() and (gvs is None or (gvs.view(np.uint8) == pvs.view(np.uint8)).all())
    rest = np.ones(pages * P, bool)
    rest[slots[~gone]] = False
    assert (gk[rest] == 0x55).all() and (gks is None or (gks.view(np.uint8)[rest] == 0x55).all())
    at = slots[~gone]
    want, err = (t[torch.from_numpy(~gone)] for t in turned(k, wk, pos, f, None, interleaved))
    if mode == "same":
        got = torch.from_numpy(gk[at].copy()).view(TDT[dt]).double()
        assert ((got - want).abs() <= rounded(want, err, dt)).all()
    else:
        _held_ok(gk[at], gks[at], want.numpy(), err.numpy(), mode, clip, dmax)
    # with nothing to turn and no norm the keys are the write's too, bit for bit
    zero = torch.zeros(T, dtype=torch.int32, device=DEV)
    fq.kv_append(cache, None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], torch.from_numpy(where).to(DEV), zero, f.to(DEV), None, None, EPS, interleaved, None, clip, dmax)
    for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (plain.k, plain.v, plain.k_scale, plain.v_scale)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_shows_what_is_not_finite():
    """A key row with a NaN or an infinity reads back as NaN, as after the cache's own write."""
    T, H, D = 5, 2, 64
    x, _ = make(T, 0, H, D, "bf16", 3)
    x[1, 0, 3], x[2, 1, 60] = math.nan, math.inf
    pos, f, slots = (t.to(DEV) for t in (torch.arange(T, dtype=torch.int32), freqs(D), torch.arange(T, dtype=torch.int32)))
    table, cu = torch.tensor([[0]], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for mode in ("int8", "e4m3", "int4"):
        cache = fq.empty_kv_cache(1, H, 16, D, mode, DEV)
        fq.kv_append(cache, None, x[:, :H].to(DEV), x[:, H:].to(DEV), slots, pos, f)
        k, v = fq.kv_read(cache, table, cu, T, torch.bfloat16)
        bad = torch.zeros(T, H, dtype=torch.bool)
        bad[1, 0] = bad[2, 1] = True
        assert torch.equal(torch.isnan(k.cpu()).all(-1), bad) and torch.equal(torch.isnan(k.cpu()).any(-1), bad)
        assert torch.isfinite(v).all()


def test_nothing_to_do():
    f = freqs(64).to(DEV)
    none, pos = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    q, k = fq.qk_rope(none, none[:, :2], pos, f)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    cache = fq.empty_kv_cache(2, 2, 16, 64, "int8", DEV)
    assert fq.kv_append(cache, none, none[:, :2], none[:, :2], pos, pos, f).shape == (0, 4, 64)


@pytest.mark.parametrize("mode", ["bf16", "int8"])
def test_captured_and_on_another_stream(mode):
    T, Hq, H, D = 40, 8, 2, 128
    x, _ = make(T, Hq, H, D, "bf16", 1)
    f = freqs(D).to(DEV)
    xd, pos, slots = x.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    cache, ref = (fq.empty_kv_cache(4, H, 16, D, mode, DEV) for _ in range(2))

    def step(c, stream=None):
        return fq.kv_append(c, xd[:, :Hq], xd[:, Hq:Hq + H], xd[:, Hq + H:], slots, pos, f, stream=stream)

    for c in (cache, ref):
        c.k.view(torch.uint8).fill_(0), c.v.view(torch.uint8).fill_(0)
        if c.k_scale is not None:
            c.k_scale.fill_(0), c.v_scale.fill_(0)
    step(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    for i in range(3):
        x2, _ = make(T, Hq, H, D, "bf16", 100 + i)
        xd.copy_(x2)
        pos.add_(17)
        want = step(ref)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8)) and torch.equal(cache.v.view(torch.uint8), ref.v.view(torch.uint8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(cache, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
