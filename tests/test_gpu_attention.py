"""GPU: attention over the paged cache and over packed prompts, against fp64 with a derived
elementwise bound (attn_ref.bound)."""
import math

import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, bound, encode, pack, softmax_attend, values
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
MODES = ["same", "int8", "e4m3", "int4", "fp4"]


def _fill(lens, H, D, P, mode, dt, seed, garbage=True, spare=2):
    """A cache holding random rows of the given lengths in shuffled pages; every other byte of codes and scales is set so
    that it reads as NaN or as large values.  Returns (cache, table, [k64], [v64])."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // P) for n in lens]
    pages = sum(held) + spare
    perm = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(lens), max(held + [1]) + 1), pages + 5, np.int32)
    m = dt if mode == "same" else mode
    cache = fq.empty_kv_cache(pages, H, P, D, m, "cpu")
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None and garbage:
            t.view(torch.uint8).fill_(0xFF)  # 16-bit, fp32, E4M3 and e8m0: NaN
    ks, vs, at = [], [], 0
    for i, n in enumerate(lens):
        table[i, :held[i]] = perm[at:at + held[i]]
        at += held[i]
        out = []
        for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            x = (torch.randn(n, H, D, generator=g) * torch.exp(0.7 * torch.randn(n, H, 1, generator=g))).to(TDT[dt])
            if mode == "same":
                c, s, val = x, None, x.double()
            else:
                code, sc = encode(x, mode)
                c, s = torch.from_numpy(pack(code, mode)), torch.from_numpy(sc if mode != "fp4" else sc.astype(np.uint8))
                val = torch.from_numpy(values(code, sc, mode))
            for t in range(n):
                p, o = int(table[i, t // P]), t % P
                if mode == "same":
                    codes[p, :, o] = c[t]
                else:
                    codes.view(torch.uint8)[p, :, o] = c[t]
                    scales[p, :, o] = s[t]
            out.append(val)
        ks.append(out[0])
        vs.append(out[1])
    dev = [None if t is None else t.to(DEV) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    return fq.KVCache(m, *dev), torch.from_numpy(table).to(DEV), ks, vs


def _check_rows(got, lse, want, dt, D, n, p_dt, label):
    out, wl, absv, top, vmax = want
    tol = bound(out, absv, top, vmax, n, D, dt, p_dt)
    err = (got.double() - out).abs()
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    say(f"[gpu]   {label}: worst error {worst:.3f} of its bound")
    assert not got.isnan().any() and (err <= tol).all(), (label, worst)
    if lse is not None:
        lt = (D + 8) * 2.0 ** -24 * top + 2.0 ** -21 * (1 + wl.abs().nan_to_num(posinf=0.0)) + math.sqrt(max(n, 1)) * 2.0 ** -23
        empty = wl == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert ((lse.double() - wl)[~empty].abs() <= lt[~empty]).all(), label


def _decode(lens, Hq, H, D, P, mode, dt, seed=0, scale=0.0, **kw):
    cache, table, ks, vs = _fill(lens, H, D, P, mode, dt, seed)
    B = len(lens)
    q = (2.0 * torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(seed + 1))).to(TDT[dt])
    lse = torch.full((B, Hq), 7.0, device=DEV)
    out = fq.attn_decode(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale, lse=lse, **kw)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    for b, n in enumerate(lens):
        want = softmax_attend(q[b:b + 1].double(), ks[b], vs[b], torch.tensor([n]), scale or 1 / math.sqrt(D))
        _check_rows(out[b:b + 1], lse[b:b + 1], want, dt, D, n, dt if mode == "same" else "f16", f"b={b} n={n}")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,H,D,P", [(4, 4, 64, 16), (8, 1, 128, 32), (14, 2, 96, 16), (3, 3, 256, 64), (20, 1, 128, 128), (16, 2, 32, 16), (5, 1, 160, 16)])
def test_decode(mode, dt, Hq, H, D, P):
    say(f"[gpu] decode {mode} {dt} Hq={Hq} H={H} D={D} P={P}")
    _decode([1, 0, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300], Hq, H, D, P, mode, dt)


@pytest.mark.parametrize("mode", MODES)
def test_decode_split_over_the_length(mode):
    say(f"[gpu] decode long {mode}")
    _decode([5000, 1, 0, 2500], 8, 2, 128, 64, mode, "bf16", seed=3)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("Hq,H,D,P", [(4, 4, 64, 16), (14, 2, 96, 16), (3, 3, 256, 64), (20, 1, 128, 128), (5, 1, 160, 16), (8, 8, 128, 32)])
def test_decode_split_with_short_sequences_between(mode, Hq, H, D, P):
    """A table too long for a workgroup a sequence: sequences of one to nineteen units, split at any place, whole ones and
    empty ones between them."""
    say(f"[gpu] decode split {mode} Hq={Hq} H={H} D={D} P={P}")
    _decode([640, 1, 0, 129, 300, 2400, 17, 128, 0, 33, 1025, 2], Hq, H, D, P, mode, "bf16", seed=11)


@pytest.mark.parametrize("mode,Hq,H,D", [("same", 8, 1, 64), ("int8", 4, 2, 128), ("int4", 3, 1, 96), ("e4m3", 17, 1, 256), ("fp4", 2, 1, 128)])
def test_decode_of_one_long_sequence(mode, Hq, H, D):
    """More parts than a join takes at once, with its elements in slices; and a batch past 64, planned by whole workgroups."""
    say(f"[gpu] decode one long {mode} Hq={Hq} H={H} D={D}")
    _decode([9001], Hq, H, D, 32, mode, "bf16", seed=13)
    _decode([4100] + [0, 3, 130] * 25, Hq, H, D, 32, mode, "f16", seed=14)


@pytest.mark.parametrize("mode,H,D", [("same", 8, 64), ("int8", 16, 128), ("e4m3", 8, 64), ("int4", 8, 128), ("fp4", 8, 32)])
@pytest.mark.parametrize("most", [1000, 1100])
def test_decode_of_many_sequences(mode, H, D, most):
    """More sequences and heads than there are CUs, below and above the length up to which each is one workgroup's."""
    say(f"[gpu] decode many {mode} H={H} D={D} most={most}")
    lens = [(most * (i * i + 1) // 1090) % (most + 1) for i in range(33)] + [most]
    _decode(lens, 2 * H, H, D, 16, mode, "f16", seed=12)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 24, 40, 112, 200])
def test_decode_odd_head_sizes(dt, D):
    for mode in ("same", "int8", "int4", "e4m3"):
        say(f"[gpu] decode {mode} {dt} D={D}")
        _decode([1, 17, 130], 6, 2, D, 16, mode, dt, seed=5)


@pytest.mark.parametrize("scale", [0.5, 4.0, -0.2])
def test_decode_scales(scale):
    for mode in ("same", "e4m3"):
        _decode([1, 40, 700], 8, 2, 64, 16, mode, "f16", seed=6, scale=scale)


def test_decode_large_and_tiny_values():
    """Scores far apart (the running maximum moves by thousands), values of very different sizes token by token."""
    B, Hq, H, D, P, n = 2, 4, 2, 64, 16, 500
    g = torch.Generator().manual_seed(9)
    for mode in ("bf16", "int8", "fp4"):
        x = torch.randn(n, H, D, generator=g) * torch.linspace(0.0, 60.0, n)[:, None, None]
        y = torch.randn(n, H, D, generator=g) * torch.exp(torch.empty(n, H, 1).uniform_(-40, 40, generator=g))
        x, y = x.bfloat16(), y.bfloat16()
        cache = fq.empty_kv_cache(-(-n // P), H, P, D, mode, DEV)
        fq.kv_write(cache, x.to(DEV), y.to(DEV), torch.arange(n, dtype=torch.int32, device=DEV))
        table = torch.arange(-(-n // P), dtype=torch.int32, device=DEV)[None].repeat(B, 1)
        lens = torch.tensor([n, n // 2], dtype=torch.int32, device=DEV)
        q = torch.randn(B, Hq, D, generator=g).bfloat16()
        out = fq.attn_decode(q.to(DEV), cache, table, lens).cpu()
        k64, v64 = (x.double(), y.double()) if mode == "bf16" else (torch.from_numpy(values(*encode(t, mode), mode)) for t in (x, y))
        for b, m in enumerate((n, n // 2)):
            want = softmax_attend(q[b:b + 1].double(), k64[:m], v64[:m], torch.tensor([m]), 1 / 8)
            _check_rows(out[b:b + 1], None, want, "bf16", D, m, "bf16" if mode == "bf16" else "f16", f"{mode} {m}")


def test_decode_leaves_out_pages_outside_the_cache():
    lens = [40]
    for mode in MODES:
        cache, table, ks, vs = _fill(lens, 2, 64, 16, mode, "bf16", 4)
        table[0, 1] = -7  # tokens 16 .. 31 are gone
        q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
        out = fq.attn_decode(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)).cpu()
        keep = [t for t in range(40) if not 16 <= t < 32]
        want = softmax_attend(q.double(), ks[0][keep], vs[0][keep], torch.tensor([24]), 1 / 8)
        _check_rows(out, None, want, "bf16", 64, 40, "bf16" if mode == "same" else "f16", mode)
        table[0] = 1 << 30
        out = fq.attn_decode(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert (out == 0).all()
    # lengths beyond the table's reach are capped at it, negative ones are 0
    cache, table, ks, vs = _fill([32], 2, 64, 16, "int8", "bf16", 4)
    q = torch.randn(1, 4, 64).bfloat16().to(DEV)
    a = fq.attn_decode(q, cache, table[:, :2], torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV))
    b = fq.attn_decode(q, cache, table[:, :2], torch.tensor([32], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b)
    assert (fq.attn_decode(q, cache, table, torch.tensor([-5], dtype=torch.int32, device=DEV)) == 0).all()
    assert (fq.attn_decode(q, cache, table[:, :0], torch.tensor([9], dtype=torch.int32, device=DEV)) == 0).all()


def test_decode_nan_reaches_only_who_sees_it():
    """A NaN key inside one sequence's length makes that sequence's rows of its heads NaN, and no other's."""
    lens = [40, 40]
    cache, table, ks, vs = _fill(lens, 2, 64, 16, "same", "bf16", 4)
    page = int(table[0, 1])
    cache.k[page, 1, 3, 5] = math.nan
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    out = fq.attn_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert out[0, 2:].isnan().all() and not out[0, :2].isnan().any() and not out[1].isnan().any()


@pytest.mark.parametrize("Hq", [2, 4, 32])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_seen_infinities_stay_infinities(dtype, Hq):
    """An infinite value that a row sees with a weight above zero makes that element infinite, not NaN, and no other element:
    with one and two heads a group, where the weights count in two parts, and with 16; in a prompt the same."""
    g = torch.Generator().manual_seed(8)
    n, H, D = 300, 2, 64
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    k, v = (torch.randn(n, H, D, generator=g).to(dt).to(DEV) for _ in range(2))
    q = torch.randn(n, Hq, D, generator=g).to(dt).to(DEV)
    v[7, 0, 3], v[290, 0, 5], v[130, 1, 60] = math.inf, -math.inf, -math.inf
    cache = fq.empty_kv_cache(20, H, 16, D, dtype, DEV)
    fq.kv_write(cache, k, v, torch.arange(n, dtype=torch.int32, device=DEV))
    table = torch.arange(20, dtype=torch.int32, device=DEV)[None]
    want = torch.zeros(Hq, D, device=DEV)
    want[: Hq // 2, 3], want[: Hq // 2, 5], want[Hq // 2 :, 60] = math.inf, -math.inf, -math.inf
    last = [fq.attn_decode(q[-1:], cache, table, torch.tensor([n], dtype=torch.int32, device=DEV))[0],
            fq.attn_prefill(q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV))[-1]]
    for got in last:
        assert torch.equal(torch.where(got.isinf(), got.float(), 0.0), want) and not got.isnan().any()


@pytest.mark.parametrize("mode", MODES[1:])
def test_decode_of_rows_that_hold_nan(mode):
    """A value row with a NaN (an infinity) written to a low-bit cache reads as NaN: per token all of its elements, per group
    its 32; a key row makes every element of its heads' outputs NaN."""
    g = torch.Generator().manual_seed(2)
    n, H, D, P = 50, 2, 128, 16
    x, y = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    y[20, 1, 70] = math.nan
    y[33, 1, 70] = math.inf
    cache = fq.empty_kv_cache(4, H, P, D, mode, DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = torch.randn(1, 4, D, generator=g).bfloat16().to(DEV)
    fq.kv_write(cache, x.to(DEV), y.to(DEV), slots)
    out = fq.attn_decode(q, cache, table, lens)[0].isnan()
    assert not out[:2].any()
    hit = torch.zeros(D, dtype=torch.bool, device=DEV)
    hit[64:96] = True
    assert (out[2:] == (hit if mode == "fp4" else True)).all()
    x[5, 0, 3] = math.nan
    fq.kv_write(cache, x.to(DEV), y.to(DEV), slots)
    assert fq.attn_decode(q, cache, table, lens)[0, :2].isnan().all()


def test_decode_repeats_bit_for_bit_and_takes_a_workspace():
    cache, table, *_ = _fill([3000, 17, 900], 2, 128, 32, "int4", "bf16", 4)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    lens = torch.tensor([3000, 17, 900], dtype=torch.int32, device=DEV)
    ws = torch.full((max(1, fq.attn_decode_workspace_size(q, cache, table)),), 0xFF, dtype=torch.uint8, device=DEV)
    a = fq.attn_decode(q, cache, table, lens)
    for _ in range(3):
        assert torch.equal(a, fq.attn_decode(q, cache, table, lens, workspace=ws))


def _prefill(lq, lk, Hq, H, D, dt, causal=True, seed=0, scale=0.0):
    g = torch.Generator().manual_seed(seed)
    cq, ck = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32), np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    q = (2.0 * torch.randn(int(cq[-1]), Hq, D, generator=g)).to(TDT[dt])
    k, v = (torch.randn(int(ck[-1]), H, D, generator=g).to(TDT[dt]) for _ in range(2))
    pad = 3  # rows past the last sequence, holding NaN: neither read nor written
    ext = lambda t: torch.cat([t, torch.full((pad, *t.shape[1:]), math.nan, dtype=t.dtype)]).to(DEV)  # noqa: E731
    qd, kd, vd = ext(q), ext(k), ext(v)
    out = torch.full_like(qd, 5.0)
    lse = torch.full((qd.shape[0], Hq), 5.0, device=DEV)
    fq.attn_prefill(qd, kd, vd, torch.from_numpy(cq).to(DEV), torch.from_numpy(ck).to(DEV), causal, scale, out, lse)
    torch.cuda.synchronize()
    assert (out[len(q):] == 5.0).all() and (lse[len(q):] == 5.0).all()
    out, lse = out.cpu(), lse.cpu()
    for b in range(len(lq)):
        a, e = cq[b], cq[b + 1]
        s = slice(ck[b], ck[b + 1])
        vis = (torch.arange(lq[b]) + lk[b] - lq[b] + 1).clamp(0, lk[b]) if causal else torch.full((lq[b],), lk[b])
        want = softmax_attend(q[a:e].double(), k[s].double(), v[s].double(), vis, scale or 1 / math.sqrt(D))
        _check_rows(out[a:e], lse[a:e], want, dt, D, lk[b], dt, f"b={b} {lq[b]} over {lk[b]}")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,H,D", [(4, 4, 64), (8, 2, 128), (6, 2, 96), (2, 1, 256), (7, 1, 128), (3, 3, 32)])
def test_prefill(dt, Hq, H, D):
    say(f"[gpu] prefill {dt} Hq={Hq} H={H} D={D}")
    lens = [1, 0, 2, 31, 33, 64, 65, 127, 128, 129, 255, 257, 300]
    _prefill(lens, lens, Hq, H, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prefill_behind_a_prefix(dt):
    say(f"[gpu] prefill prefix {dt}")
    _prefill([1, 5, 64, 130, 200, 3], [300, 5, 190, 131, 777, 64], 4, 2, 128, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prefill_not_causal_and_short_keys(dt):
    say(f"[gpu] prefill full {dt}")
    _prefill([1, 5, 64, 130, 200, 3], [300, 0, 190, 7, 777, 1], 4, 2, 64, dt, causal=False)
    # fewer keys than rows: the first rows see nothing and give zeros
    _prefill([10, 200, 3, 300, 140], [4, 70, 0, 299, 1], 4, 2, 64, dt)


@pytest.mark.parametrize("D", [8, 16, 40, 72, 104, 200])
def test_prefill_odd_head_sizes(D):
    for dt in ("bf16", "f16"):
        _prefill([1, 77, 140], [1, 77, 200], 4, 2, D, dt, seed=2)


def test_prefill_long():
    _prefill([1500, 3], [1500, 3], 2, 1, 128, "bf16", seed=4)
    _prefill([1300], [1300], 2, 2, 64, "f16", seed=5, scale=1.0)


@pytest.mark.parametrize("lq,lk", [([40], [5000]), ([130, 1, 300, 0], [2100, 3000, 1300, 20]), ([1500], [1500])])
def test_prefill_split_over_the_keys(lq, lk):
    """Few rows over many keys: the walks are cut into parts and joined."""
    for dt, D in (("bf16", 128), ("f16", 64), ("bf16", 200)):
        q, k = torch.empty(sum(lq), 4, D, device=DEV), torch.empty(sum(lk), 2, D, device=DEV)
        assert fq.attn_prefill_workspace_size(q, k, torch.empty(len(lq) + 1, device=DEV)) > 0
        _prefill(lq, lk, 4, 2, D, dt, seed=6)


def test_prefill_many_sequences():
    """More sequences than a wave has lanes."""
    rng = np.random.default_rng(8)
    lens = [int(n) for n in rng.integers(0, 9, 150)] + [200, 0, 130]
    _prefill(lens, lens, 2, 1, 64, "bf16", seed=7)


def test_prefill_large_scores():
    """Scores whose maximum moves by hundreds between key tiles, upwards and downwards."""
    g = torch.Generator().manual_seed(3)
    L, Hq, D = 600, 2, 64
    ramp = torch.cat([torch.linspace(0, 40, L // 2), torch.linspace(40, 0, L // 2)])[:, None, None]
    q = torch.randn(L, Hq, D, generator=g).bfloat16()
    k = (torch.randn(L, Hq, D, generator=g) * ramp).bfloat16()
    v = torch.randn(L, Hq, D, generator=g).bfloat16()
    cu = torch.tensor([0, L], dtype=torch.int32, device=DEV)
    out = fq.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu).cpu()
    want = softmax_attend(q.double(), k.double(), v.double(), torch.arange(L) + 1, 1 / 8)
    _check_rows(out, None, want, "bf16", D, L, "bf16", "ramp")


def test_prefill_strided_rows_of_a_fused_projection():
    g = torch.Generator().manual_seed(4)
    L, Hq, H, D = 150, 4, 2, 128
    qkv = torch.randn(L, Hq + 2 * H, D, generator=g).bfloat16()
    cu = torch.tensor([0, 100, L], dtype=torch.int32, device=DEV)
    d = qkv.to(DEV)
    q, k, v = d[:, :Hq], d[:, Hq:Hq + H], d[:, Hq + H:]
    wide = torch.zeros(L, Hq + 1, D, dtype=torch.bfloat16, device=DEV)
    fq.attn_prefill(q, k, v, cu, out=wide[:, :Hq])
    a = fq.attn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(wide[:, :Hq], a) and (wide[:, Hq] == 0).all()
    # heads outermost in memory
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    assert torch.equal(fq.attn_prefill(qh, kh, vh, cu), a)


@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("lq,lk", [([3], [20000]), ([1, 130, 2], [17000, 300, 9]), ([40], [600]), ([0, 150, 1], [0, 100, 4100])])
def test_prefill_few_rows_behind_many_keys(lq, lk, D):
    """Walks cut into up to 32 parts of 8 tiles and joined, with short and empty ones, and rows that see nothing, beside them."""
    say(f"[gpu] prefill {lq} over {lk} D={D}")
    _prefill(lq, lk, 4, 2, D, "bf16", seed=9)
    _prefill(lq, lk, 3, 1, D, "f16", seed=10)
    _prefill(lq, lk, 4, 2, D, "f16", causal=False, seed=11)


def test_prefill_future_infinities_and_nan_stay_hidden():
    """Keys and values after a row, and other sequences' rows, never reach it, whatever they hold."""
    g = torch.Generator().manual_seed(5)
    L, H, D = 200, 2, 64
    q, k, v = (torch.randn(L, H, D, generator=g).bfloat16().to(DEV) for _ in range(3))
    cu = torch.tensor([0, 90, L], dtype=torch.int32, device=DEV)
    a = fq.attn_prefill(q, k, v, cu)
    k[50], v[50], k[150, :, 3], v[199] = math.nan, math.inf, -math.inf, math.nan
    b = fq.attn_prefill(q, k, v, cu)
    for s in (slice(0, 50), slice(90, 150)):
        assert torch.equal(a[s], b[s])
    assert b[50:90].isnan().all() and b[199].isnan().all()


def test_nothing_to_do():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert fq.attn_prefill(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), cu).shape == (0, 4, 64)
    out = fq.attn_prefill(torch.ones(4, 4, 64, dtype=torch.bfloat16, device=DEV), e(0, 2, 64), e(0, 2, 64),
                          torch.tensor([0, 4], dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV))
    assert (out == 0).all()
    cache = fq.empty_kv_cache(2, 2, 16, 64, "int8", DEV)
    assert fq.attn_decode(e(0, 4, 64), cache, torch.empty(0, 2, dtype=torch.int32, device=DEV),
                          torch.empty(0, dtype=torch.int32, device=DEV)).shape == (0, 4, 64)
    torch.cuda.synchronize()
