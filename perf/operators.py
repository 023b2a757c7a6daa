"""Cases and plain forms of the attention operators: the paged key-value cache (written, low-bit
codes included, and read back), attention of one new token over it, and causal attention over
packed prompts.

A cache holds pages of `page` tokens: codes [pages, heads, page, D] (two codes a byte for the 4-bit
modes) and, for the low-bit modes, one fp32 scale per (page, head, token) or, for `fp4`, one e8m0
byte per 32 elements.  Modes: "same" (the inputs' own 16-bit type), "int8", "e4m3", "int4", "fp4".

With `own` false, run() is elementary torch operations in fp32, rounded once at the end; with
`own` true, the package's operators.  exact() is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _device():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


# ---- the cases ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence early in its answer: its newest token written, its short context read back
        dict(name="cache_token", op="cache", mode="int8", dtype="bf16", B=1, ctx=33, new=1, spread=1.0, Hkv=8, D=128, page=16),
        # a chunk of six prompts of uneven length written, and their whole contexts read for the chunk's attention
        dict(name="cache_chunk", op="cache", mode="int4", dtype="bf16", B=6, ctx=9001, new=512, spread=12.0, Hkv=8, D=128, page=64),
        # the same for sixteen long documents, in the per-group 4-bit format
        dict(name="cache_long", op="cache", mode="fp4", dtype="bf16", B=16, ctx=32768, new=2048, spread=8.0, Hkv=8, D=128, page=32),
        # one user's first words: latency only
        dict(name="decode_one", op="decode", mode="same", dtype="bf16", B=1, ctx=77, spread=1.0, idle=0, append=False,
             Hq=32, Hkv=8, D=128, page=16),
        # a step of a running batch, 16-bit cache: the new keys and values written, then attended
        dict(name="decode_step", op="decode", mode="same", dtype="bf16", B=32, ctx=4096, spread=30.0, idle=0, append=True,
             Hq=32, Hkv=8, D=128, page=16),
        # two long documents: few rows, the cache's length has to be split
        dict(name="decode_long", op="decode", mode="int8", dtype="bf16", B=2, ctx=131072, spread=1.5, idle=0, append=False,
             Hq=64, Hkv=8, D=128, page=128),
        # a full server at the hidden size 8192 (64 heads of 128), int4 cache
        dict(name="decode_many", op="decode", mode="int4", dtype="bf16", B=128, ctx=16384, spread=16.0, idle=0, append=False,
             Hq=64, Hkv=8, D=128, page=64),
        # a batch captured at a fixed size with idle places (length 0), heads of 64 without sharing, fp8 cache
        dict(name="decode_idle", op="decode", mode="e4m3", dtype="f16", B=37, ctx=2000, spread=50.0, idle=5, append=False,
             Hq=16, Hkv=16, D=64, page=32),
        # seven short questions packed into one call
        dict(name="prefill_short", op="prefill", dtype="f16", B=7, most=200, prefix=0, spread=40.0, Hq=16, Hkv=16, D=64),
        # nine prompts of uneven length packed, grouped heads
        dict(name="prefill_packed", op="prefill", dtype="bf16", B=9, most=4096, prefix=0, spread=20.0, Hq=32, Hkv=8, D=128),
        # chunks of four long prompts, each behind the part already in the cache
        dict(name="prefill_chunk", op="prefill", dtype="f16", B=4, most=1024, prefix=8192, spread=4.0, Hq=32, Hkv=8, D=128),
        # one long document on one of eight cards that share 64 heads
        dict(name="prefill_long", op="prefill", dtype="bf16", B=1, most=32768, prefix=0, spread=1.0, Hq=8, Hkv=1, D=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "decode", "prefill"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), spread=round(rng.uniform(1.0, 40.0), 2))
    D = rng.choice([64, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 8, 16])
    if op == "cache":
        c.update(mode=rng.choice(["same", "int8", "e4m3", "int4", "fp4"]), B=_spread(rng, 1, 64), new=_spread(rng, 1, 2048),
                 Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]))
        c["ctx"] = _spread(rng, 4, max(8, min(32768, (16 * 32768 * 8 * 128) // (2 * c["B"] * Hkv * D))))
    elif op == "decode":
        c.update(mode=rng.choice(["same", "int8", "e4m3", "int4", "fp4"]), B=_spread(rng, 1, 128),
                 idle=rng.choice([0, 0, 1, 3]), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), D=D,
                 page=rng.choice([16, 32, 64, 128]))
        c["append"] = c["mode"] == "same" and rng.random() < 0.5
        c["ctx"] = _spread(rng, 4, max(8, min(131072, (128 * 16384 * 8 * 128) // (4 * c["B"] * Hkv * D))))
    else:
        c.update(B=_spread(rng, 1, 24), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), D=D)
        c["prefix"] = 0 if rng.random() < 0.7 else _spread(rng, 1, 4096)
        room = 32768 ** 2 * 8 * 128 / (4.0 * c["B"] * c["Hq"] * D)  # padded scores x D, well below the longest listed prompt's
        p = c["prefix"]
        c["most"] = _spread(rng, 4, max(8, min(16384, int(math.sqrt(room + 0.25 * p * p) - 0.5 * p))))
    return c


def _lengths(n, most, spread):
    """n lengths from `most` down to about most / spread, evenly on a log scale, in a mixed order."""
    return [max(1, int(round(most * spread ** -((i * 0.6180339887498949) % 1.0)))) for i in range(n)]


def _contexts(case):
    """Tokens in the cache of each sequence, the newest included; a decode batch's idle places hold none."""
    lens = _lengths(case["B"], case["ctx"], case["spread"])
    for i in range(min(case.get("idle", 0), case["B"] - 1)):
        lens[1 + (2 * i) % (case["B"] - 1)] = 0
    return lens


def _prompts(case):
    q = _lengths(case["B"], case["most"], case["spread"])
    p = _lengths(case["B"], case["prefix"], case["spread"])[::-1] if case["prefix"] else [0] * case["B"]
    return q, [a + b for a, b in zip(q, p)]


def _token_bytes(case):
    """Bytes of one token's key (or value) of one head in the cache, scale included."""
    D = case["D"]
    return {"same": 2 * D, "int8": D + 4, "e4m3": D + 4, "int4": D // 2 + 4, "fp4": D // 2 + 2 * (-(-D // 64))}[case["mode"]]


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "cache":
        lens = _contexts(case)
        new = sum(min(case["new"], n) for n in lens)
        row = 2 * Hkv * D * 2  # a token's keys and values in 16 bits
        held = 2 * Hkv * _token_bytes(case)
        return {"bytes": new * (row + held + 4) + (sum(lens) - new) * held + sum(lens) * row,
                "flops": 2 * 2 * Hkv * D * (new + sum(lens))}
    if case["op"] == "decode":
        lens = _contexts(case)
        held, rows = 2 * Hkv * _token_bytes(case), 2 * case["B"] * case["Hq"] * D * 2
        new = sum(n > 0 for n in lens) * (2 * Hkv * D * 2 + held) if case["append"] else 0
        old = sum(lens) - (sum(n > 0 for n in lens) if case["append"] else 0)
        return {"bytes": old * held + rows + new, "flops": 4 * sum(lens) * case["Hq"] * D}
    q, k = _prompts(case)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, k))
    return {"bytes": 2 * D * (2 * sum(q) * case["Hq"] + 2 * sum(k) * Hkv), "flops": 4 * pairs * case["Hq"] * D}


# ---- inputs ------------------------------------------------------------------------------

def _normal(shape, gen, dtype, channels=None):
    x = torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (x if channels is None else x * channels).to(dtype)


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _empty_cache(case, pages, dev):
    """[codes, scales] of one side of the cache; scales None in 16 bits."""
    h, p, D, mode = case["Hkv"], case["page"], case["D"], case["mode"]
    if mode == "same":
        return [torch.zeros(pages, h, p, D, dtype=DTYPES[case["dtype"]], device=dev), None]
    code = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(mode, torch.uint8)
    codes = torch.zeros(pages, h, p, D if mode in ("int8", "e4m3") else D // 2, dtype=torch.uint8, device=dev).view(code)
    if mode == "fp4":
        return [codes, torch.zeros(pages, h, p, 2 * (-(-D // 64)), dtype=torch.uint8, device=dev)]
    return [codes, torch.zeros(pages, h, p, dtype=torch.float32, device=dev)]


def prepare(case, seed):
    dev, dt = _device(), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    Hkv, D = case["Hkv"], case["D"]
    # a few channels of the keys stand out, as they do in a trained model
    wide = torch.where(torch.rand(Hkv, D, generator=gen, device=dev) < 0.02, 8.0, 1.0)
    s = dict(case=case)
    if case["op"] == "prefill":
        q, k = _prompts(case)
        s.update(cu_q=_ints([0, *np.cumsum(q).tolist()], dev), cu_k=_ints([0, *np.cumsum(k).tolist()], dev), max_q=max(q), max_k=max(k),
                 q=_normal((sum(q), case["Hq"], D), gen, dt), k=_normal((sum(k), Hkv, D), gen, dt, wide),
                 v=_normal((sum(k), Hkv, D), gen, dt))
        return s
    lens, page = _contexts(case), case["page"]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    places = host.permutation(pages)[:sum(held)].astype(np.int32)
    table = np.full((len(lens), max(1, max(held))), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = places[at:at + n]
        at += n
    kc, vc = _empty_cache(case, pages, dev), _empty_cache(case, pages, dev)
    step = max(1, (1 << 26) // (Hkv * page * D))
    for side, ch in ((kc, wide[:, None, :]), (vc, None)):
        for a in range(0, pages, step):
            b = min(pages, a + step)
            codes, scales = _encode(_normal((b - a, Hkv, page, D), gen, dt, ch), case["mode"])
            side[0][a:b] = codes
            if scales is not None:
                side[1][a:b] = scales
    s.update(k_cache=kc[0], k_scale=kc[1], v_cache=vc[0], v_scale=vc[1], table=torch.from_numpy(table).to(dev))
    new = [min(case["new"], n) for n in lens] if case["op"] == "cache" else [min(1, n) if case["append"] else 0 for n in lens]
    slots = [int(table[i, t // page]) * page + t % page for i, n in enumerate(lens) for t in range(n - new[i], n)]
    if case["op"] == "cache" or case["append"]:
        s.update(slots=_ints(slots, dev), k=_normal((sum(new), Hkv, D), gen, dt, wide), v=_normal((sum(new), Hkv, D), gen, dt))
    if case["op"] == "cache":
        s.update(cu=_ints([0, *np.cumsum(lens).tolist()], dev), total=sum(lens))
    else:
        s.update(lengths=_ints(lens, dev), max_length=max(lens), q=_normal((len(lens), case["Hq"], D), gen, dt))
    return s


# ---- the plain form: elementary torch operations in fp32 ------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x, mode):
    """Codes and scales of rows [..., D]: scale = max|x| / qmax in fp32 and code = x / scale rounded half to even;
    for fp4 per group of 32 the power of two floor(log2 max) - 2."""
    if mode == "same":
        return x, None
    x = x.float()
    if mode == "fp4":
        g = x.unflatten(-1, (-1, 32))
        top = g.abs().amax(-1)
        e8 = torch.where(top > 0, torch.frexp(top).exponent + 124, 0).clamp_(0, 254)
        a = torch.ldexp(g, (127 - e8).unsqueeze(-1)).flatten(-2)
        neg, a = torch.signbit(a), a.abs()
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)) | (neg.to(torch.uint8) << 3)
        e8 = e8.to(torch.uint8)
        if e8.shape[-1] % 2:
            e8 = torch.cat([e8, torch.zeros_like(e8[..., :1])], -1)
        return code[..., 0::2] | (code[..., 1::2] << 4), e8
    scale = x.abs().amax(-1)
    scale = scale / torch.full_like(scale, QMAX[mode])  # (a division by a number would become a product with its reciprocal)
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    if mode == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale
    if mode == "int8":
        return y.round().clamp(-127.0, 127.0).to(torch.int8), scale
    n = y.round().clamp(-8.0, 7.0).to(torch.int8).view(torch.uint8) & 15
    return n[..., 0::2] | (n[..., 1::2] << 4), scale


def _decode(codes, scales, mode):
    """fp32 values of codes and scales."""
    if mode == "same":
        return codes.float()
    if mode in ("int8", "e4m3"):
        return codes.float() * scales[..., None]
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    if mode == "int4":
        return ((n ^ 8).to(torch.int8) - 8).float() * scales[..., None]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    g = table[n.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(g, (scales[..., :g.shape[-2]].int() - 127).unsqueeze(-1)).flatten(-2)


def _gather(s, at, pos):
    """Keys and values [*pos.shape, heads, D] of sequences `at` at positions `pos`, in fp32."""
    page = s["case"]["page"]
    p, o, mode = s["table"][at, pos // page].clamp(min=0).long(), pos % page, s["case"]["mode"]
    pick = lambda t: None if t is None else t[p, :, o]  # noqa: E731
    if mode == "e4m3":  # (indexed as bytes)
        codes = [s[n].view(torch.uint8)[p, :, o].view(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")]
    else:
        codes = [pick(s["k_cache"]), pick(s["v_cache"])]
    return _decode(codes[0], pick(s["k_scale"]), mode), _decode(codes[1], pick(s["v_scale"]), mode)


def _write(s):
    page, mode = s["case"]["page"], s["case"]["mode"]
    p, o = (s["slots"] // page).long(), (s["slots"] % page).long()
    for new, codes, scales in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        c, sc = _encode(new, mode)
        if mode == "e4m3":
            codes, c = codes.view(torch.uint8), c.view(torch.uint8)
        codes[p, :, o] = c
        if sc is not None:
            scales[p, :, o] = sc


def _attend(q, k, v, visible):
    """Softmax attention of q [B, Lq, Hq, D] over k, v [B, Lk, Hkv, D] where visible [B, Lq, Lk]; rows that see nothing give 0."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    q = q.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    p = torch.matmul(q * (1.0 / math.sqrt(D)), k.permute(0, 2, 3, 1).contiguous()).view(B, Hkv, -1, Lq, Lk)
    p.masked_fill_(~visible[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, Lk), v.permute(0, 2, 1, 3).contiguous()).view(B, Hkv, -1, Lq, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D)


def _rows(cu, total):
    """(sequence, position) of each packed row."""
    t = torch.arange(total, device=cu.device, dtype=torch.int32)
    b = torch.bucketize(t, cu[1:], right=True)
    return b, t - cu[b]


def _padded(x, cu, most):
    t = torch.arange(most, device=cu.device)
    inside = t < (cu[1:] - cu[:-1])[:, None]
    rows = x[(cu[:-1, None] + t).clamp_(max=x.shape[0] - 1)].float()
    return torch.where(inside[..., None, None], rows, 0.0), inside


def _plain(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if case["op"] == "cache":
        _write(s)
        k, v = _gather(s, *_rows(s["cu"], s["total"]))
        return k.to(dt), v.to(dt)
    if case["op"] == "decode":
        if case["append"]:
            _write(s)
        t = torch.arange(s["max_length"], device=s["q"].device)
        k, v = _gather(s, torch.arange(s["q"].shape[0], device=t.device)[:, None], t[None])
        inside = t < s["lengths"][:, None]
        v = torch.where(inside[..., None, None], v, 0.0)
        o = _attend(s["q"].float()[:, None], k, v, inside[:, None])[:, 0].to(dt)
        return (o, s["k_cache"], s["v_cache"]) if case["append"] else o
    q, _ = _padded(s["q"], s["cu_q"], s["max_q"])
    k, there = _padded(s["k"], s["cu_k"], s["max_k"])
    v, _ = _padded(s["v"], s["cu_k"], s["max_k"])
    before = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])  # tokens ahead of the first row
    i, j = torch.arange(s["max_q"], device=q.device), torch.arange(s["max_k"], device=q.device)
    visible = there[:, None] & (j <= (before[:, None] + i)[..., None])
    return _attend(q, k, v, visible)[_rows(s["cu_q"], s["q"].shape[0])].to(dt)


# ---- one pass --------------------------------------------------------------------------------

def _own(s):
    import flatquant_transform_quant_amd as fq

    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if case["op"] == "prefill":
        return fq.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside the tensors
        mode = case["dtype"] if case["mode"] == "same" else case["mode"]
        cache = s["cache"] = fq.KVCache(mode, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if case["op"] == "cache":
        fq.kv_write(cache, s["k"], s["v"], s["slots"])
        return fq.kv_read(cache, s["table"], s["cu"], s["total"], dt)
    if case["append"]:
        fq.kv_write(cache, s["k"], s["v"], s["slots"])
        return fq.attn_decode(s["q"], cache, s["table"], s["lengths"]), s["k_cache"], s["v_cache"]
    return fq.attn_decode(s["q"], cache, s["table"], s["lengths"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in fp64, sequence by sequence ---------------------------------------------

def _magnitudes(mode):
    """The values of the non-negative codes of a 4- or 8-bit float, by code."""
    ebits, mbits, bias = (4, 3, 7) if mode == "e4m3" else (2, 1, 1)
    out = []
    for c in range(1 << (ebits + mbits)):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        out.append(math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp((1 << mbits) + m, e - bias - mbits))
    return out[:127] if mode == "e4m3" else out


def _nearest(y, mode):
    """The value of `mode` nearest each y (fp64), ties to the even code."""
    mags = torch.tensor(_magnitudes(mode), dtype=torch.float64, device=y.device)
    mids = (mags[1:] + mags[:-1]) / 2
    a = y.abs().contiguous()
    lo, hi = torch.searchsorted(mids, a), torch.searchsorted(mids, a, right=True)
    return torch.copysign(mags[torch.where(lo % 2 == 0, lo, hi)], y)


def _held64(x, mode):
    """The fp64 values that rows x stand for once written in `mode`; the scale and the quotient that is rounded to a code are
    fp32 numbers by the format's definition (or powers of two), so that a quotient at a tie is the same tie for everybody."""
    x = x.double()
    if mode == "same":
        return x
    if mode == "fp4":
        g = x.reshape(*x.shape[:-1], -1, 32)
        top = g.abs().amax(-1, keepdim=True)
        unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(-127, 127))
        return (_nearest(g / unit, mode) * unit).reshape(x.shape)
    scale = (x.abs().amax(-1, keepdim=True) / QMAX[mode]).float().double()
    y = torch.where(scale > 0, x / scale.clamp(min=1e-300), 0.0).float().double()
    q = _nearest(y, mode) if mode == "e4m3" else y.round().clamp(-8.0 if mode == "int4" else -127.0, QMAX[mode])
    return q * scale


def _values64(codes, scales, mode):
    if mode == "same":
        return codes.double()
    raw = codes.view(torch.uint8).int()
    if mode in ("int4", "fp4"):
        raw = torch.stack([raw % 16, raw // 16], -1).reshape(*raw.shape[:-1], 2 * raw.shape[-1])
    if mode in ("int8", "int4"):
        bits = 8 if mode == "int8" else 4
        q = torch.where(raw >= 1 << (bits - 1), raw - (1 << bits), raw).double()
    else:
        m = _magnitudes(mode) + ([math.nan] if mode == "e4m3" else [])
        q = torch.tensor(m + [-v for v in m], dtype=torch.float64, device=raw.device)[raw]
    if mode == "fp4":
        unit = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
        return q * unit[..., :q.shape[-1]]
    return q * scales.double()[..., None]


def _sequence64(s, i, n):
    """Keys and values [n, heads, D] of sequence i's first n tokens, as the cache holds them."""
    page, mode = s["case"]["page"], s["case"]["mode"]
    pages = s["table"][i, :-(-n // page)].long()
    out = []
    for side in ("k", "v"):
        sc = s[side + "_scale"]
        x = _values64(s[side + "_cache"].view(torch.uint8 if mode != "same" else s[side + "_cache"].dtype)[pages],
                      None if sc is None else sc[pages], mode)
        out.append(x.transpose(1, 2).reshape(len(pages) * page, x.shape[1], x.shape[3])[:n])
    return out


def _attend64(q, k, v, before):
    """One sequence: q [Lq, Hq, D], k, v [Lk, Hkv, D]; row i sees the keys up to before + i."""
    Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[:2]
    o = torch.zeros(Lq, Hq, D, dtype=torch.float64, device=q.device)
    j = torch.arange(Lk, device=q.device)
    for a in range(0, Lq, 2048):
        b = min(Lq, a + 2048)
        last = min(Lk, before + b)
        if last <= 0:
            continue
        hidden = j[None, :last] > before + torch.arange(a, b, device=q.device)[:, None]
        for h in range(Hq):
            kh, vh = k[:last, h * Hkv // Hq], v[:last, h * Hkv // Hq]
            p = torch.softmax((q[a:b, h] @ kh.T / math.sqrt(D)).masked_fill_(hidden, -math.inf), -1)
            o[a:b, h] = torch.nan_to_num(p) @ vh if before + a < 0 else p @ vh
    return o


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        if work(case)["flops"] > 4e13:
            return None
        out, q, k = [], s["cu_q"].tolist(), s["cu_k"].tolist()
        for i in range(case["B"]):
            a, b, c, d = q[i], q[i + 1], k[i], k[i + 1]
            out.append(_attend64(s["q"][a:b].double(), s["k"][c:d].double(), s["v"][c:d].double(), (d - c) - (b - a)))
        return torch.cat(out)
    lens = _contexts(case)
    out_k, out_v, out, at = [], [], [], 0
    for i, n in enumerate(lens):
        k, v = _sequence64(s, i, n)
        new = min(case["new"], n) if case["op"] == "cache" else int(case["append"] and n > 0)
        if new:
            k[n - new:] = _held64(s["k"][at:at + new], case["mode"])
            v[n - new:] = _held64(s["v"][at:at + new], case["mode"])
            at += new
        if case["op"] == "cache":
            out_k.append(k)
            out_v.append(v)
        else:
            out.append(_attend64(s["q"][i:i + 1].double(), k, v, n - 1))
    if case["op"] == "cache":
        return torch.cat(out_k), torch.cat(out_v)
    return (torch.cat(out), None, None) if case["append"] else torch.cat(out)
