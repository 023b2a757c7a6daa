"""Cases and plain forms of more operators around the quantizer's attention layer: query and key
norms with the position rotation (`rope`), the same with keys and values appended to the paged
cache (`append`), attention of new tokens over the paged cache with a sliding window and first
tokens that stay visible (`chunk`), and the product of 8-bit codes with their scales (`gemm`).

A cache holds pages of `page` tokens: codes [pages, heads, page, D] (two codes a byte for the 4-bit
modes) and, for the low-bit modes, one fp32 scale per (page, head, token) or, for `fp4`, one e8m0
byte per 32 elements.  Modes: "same" (the inputs' own 16-bit type), "int8", "e4m3", "int4", "fp4".

With `own` false, run() is elementary torch operations in fp32 (angles, and sums of products of
codes, which pass 2^24, in fp64), rounded once at the end; with `own` true, the package's operators.
exact() is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _device():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


# ---- the cases ---------------------------------------------------------------------------

def listed():
    return [
        # three users' newest tokens between the projection and the cache: latency only
        dict(name="rope_step", op="rope", dtype="bf16", T=3, Hq=32, Hkv=8, D=128, R=128, norm=True, turn=False, axes=1, start=4000),
        # long prompts packed, at the hidden size 8192 (64 heads of 128)
        dict(name="rope_prompt", op="rope", dtype="f16", T=16384, Hq=64, Hkv=8, D=128, R=128, norm=True, turn=False, axes=1, start=0),
        # frames of a video: three axes dealt to the pairs by turns, heads of 80, no norms, pairs side by side
        dict(name="rope_video", op="rope", dtype="bf16", T=5003, Hq=16, Hkv=16, D=80, R=80, norm=False, turn=True, axes=3, start=7),
        # a step of a running batch: 48 newest tokens into an fp8 cache
        dict(name="append_step", op="append", mode="e4m3", dtype="bf16", T=48, Hq=64, Hkv=8, D=128, R=128, norm=True, turn=False,
             axes=1, start=100000, page=16),
        # packed prompts into an fp8 cache, heads of 64 with half of each rotated, some rows padding
        dict(name="append_prompt", op="append", mode="e4m3", dtype="f16", T=7777, Hq=32, Hkv=8, D=64, R=32, norm=False, turn=False,
             axes=1, start=0, page=64),
        # drafted tokens checked: five new ones each behind long contexts, int8 cache
        dict(name="chunk_verify", op="chunk", mode="int8", dtype="bf16", B=24, new=5, ctx=16384, spread=12.0, Hq=64, Hkv=8, D=128,
             page=64, window=0, sinks=0),
        # single tokens of a running batch with a window and four tokens that stay, 16-bit cache
        dict(name="chunk_step", op="chunk", mode="same", dtype="bf16", B=32, new=1, ctx=32768, spread=40.0, Hq=32, Hkv=8, D=128,
             page=16, window=1024, sinks=4),
        # chunks of five prompts of uneven length behind what the int4 cache holds of them
        dict(name="chunk_prompts", op="chunk", mode="int4", dtype="bf16", B=5, new=1024, ctx=9216, spread=6.0, Hq=32, Hkv=8, D=128,
             page=32, window=0, sinks=0),
        # one long document on one of eight cards that share 64 heads, with a window and first tokens that stay
        dict(name="chunk_document", op="chunk", mode="same", dtype="f16", B=1, new=16384, ctx=16384, spread=1.0, Hq=8, Hkv=1, D=128,
             page=128, window=4096, sinks=16),
        # four users' next tokens through the fused projection at the hidden size 8192 (64 + 2 x 8 heads of 128)
        dict(name="gemm_step", op="gemm", dtype="bf16", T=4, O=10240, H=8192),
        # a batch of odd size
        dict(name="gemm_batch", op="gemm", dtype="f16", T=333, O=8200, H=4112),
        # packed prompts at the hidden size 8192
        dict(name="gemm_prompt", op="gemm", dtype="bf16", T=8192, O=8192, H=8192),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "gemm"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    D, Hkv = rng.choice([64, 80, 128, 128, 256]), rng.choice([1, 2, 3, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    if op == "gemm":
        c.update(dtype=rng.choice(["bf16", "f16", "f32"]), T=_spread(rng, 1, 8192), O=_spread(rng, 64, 16384), H=16 * _spread(rng, 4, 1024))
        c["T"] = max(1, min(c["T"], 8192 ** 3 // (2 * c["O"] * c["H"])))
        return c
    if op in ("rope", "append"):
        c.update(T=max(1, min(_spread(rng, 1, 16384), 16384 * 72 * 128 // (2 * (Hq + Hkv) * D))), Hq=Hq, Hkv=Hkv, D=D,
                 R=rng.choice([D, D, D // 2]), norm=rng.random() < 0.6, turn=rng.random() < 0.3, axes=rng.choice([1, 1, 1, 2, 3]),
                 start=rng.choice([0, _spread(rng, 1, 1 << 20)]))
        if op == "append":
            c.update(mode=rng.choice(["same", "int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]))
        return c
    D = rng.choice([64, 96, 128, 128, 256])
    c.update(mode=rng.choice(["same", "int8", "e4m3", "int4", "fp4"]), B=_spread(rng, 1, 64), spread=round(rng.uniform(1.0, 40.0), 2),
             Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _spread(rng, 1, 8192)]), sinks=rng.choice([0, 4, 33]))
    c["new"] = 1 if rng.random() < 0.3 else _spread(rng, 1, 2048)
    # padded scores x D stay well below the document's, and the cache below the checked drafts'
    most = min(16384 ** 2 * 8 * 128 / (4.0 * c["B"] * Hq * D * c["new"]), 24 * 16384 * 8 * 128 / (2.0 * c["B"] * Hkv * D), 65536.0)
    c["ctx"] = _spread(rng, 4, max(8, int(most)))
    c["new"] = min(c["new"], c["ctx"])
    return c


def _lengths(n, most, spread):
    """n lengths from `most` down to about most / spread, evenly on a log scale, in a mixed order."""
    return [max(1, int(round(most * spread ** -((i * 0.6180339887498949) % 1.0)))) for i in range(n)]


def _token_bytes(mode, D):
    """Bytes of one token's key (or value) of one head in the cache, scale included."""
    return {"same": 2 * D, "int8": D + 4, "e4m3": D + 4, "int4": D // 2 + 4, "fp4": D // 2 + 2 * (-(-D // 64))}[mode]


def _seen(case):
    """(pairs that are seen, keys that some row sees) of the chunk case, over all sequences."""
    pairs = keys = 0
    for n in _lengths(case["B"], case["ctx"], case["spread"]):
        new, w, s = min(case["new"], n), case["window"], case["sinks"]
        last = np.arange(n - new, n, dtype=np.int64)  # each row's own position
        if w == 0:
            pairs += int((last + 1).sum())
            keys += n
        else:
            lo = np.maximum(0, last - w + 1)
            pairs += int((last - lo + 1 + np.minimum(lo, s)).sum())
            keys += n - int(lo[0]) + min(int(lo[0]), s)
    return pairs, keys


def work(case):
    if case["op"] == "gemm":
        T, O, H = case["T"], case["O"], case["H"]
        return {"bytes": T * H + O * H + 4 * (T + O) + T * O * (4 if case["dtype"] == "f32" else 2), "flops": 2 * T * O * H}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "chunk":
        pairs, keys = _seen(case)
        rows = sum(min(case["new"], n) for n in _lengths(case["B"], case["ctx"], case["spread"]))
        return {"bytes": keys * 2 * Hkv * _token_bytes(case["mode"], D) + 2 * rows * Hq * D * 2, "flops": 4 * pairs * Hq * D}
    T, extra = case["T"], 4 * case["axes"] + (4 if case["op"] == "append" else 0)
    flops = T * (Hq + Hkv) * ((4 * D if case["norm"] else 0) + 3 * case["R"])
    if case["op"] == "rope":
        return {"bytes": T * (2 * (Hq + Hkv) * D * 2 + extra), "flops": flops}
    read_back = 2 * Hkv * (_token_bytes(case["mode"], D) + 2 * D) if case["mode"] == "int8" else 0
    return {"bytes": T * (2 * Hq * D * 2 + 2 * Hkv * (2 * D + _token_bytes(case["mode"], D)) + extra + read_back),
            "flops": flops + 4 * T * Hkv * D}


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


def _prepare_gemm(case, gen, dev):
    def side(rows):
        codes = torch.empty(rows, case["H"], dtype=torch.int8, device=dev)
        step = max(1, (1 << 26) // case["H"])
        for a in range(0, rows, step):
            b = min(rows, a + step)
            codes[a:b] = (torch.randn(b - a, case["H"], generator=gen, device=dev) * 30.0).round_().clamp_(-127, 127)
        return codes, torch.exp(torch.randn(rows, generator=gen, device=dev)) * 0.01

    (a, sa), (w, sw) = side(case["T"]), side(case["O"])
    return dict(case=case, a=a, a_scale=sa, w=w, w_scale=sw)


def _prepare_rows(case, gen, host, dev):
    dt, T, Hkv, D, half = DTYPES[case["dtype"]], case["T"], case["Hkv"], case["D"], case["R"] // 2
    # the rows as a fused projection leaves them: queries, keys and values of a token side by side
    wide = torch.where(torch.rand(case["Hq"] + 2 * Hkv, D, generator=gen, device=dev) < 0.02, 6.0, 1.0)
    qkv = _normal((T, case["Hq"] + 2 * Hkv, D), gen, dt, wide)
    s = dict(case=case, q=qkv[:, :case["Hq"]], k=qkv[:, case["Hq"]:case["Hq"] + Hkv], q_weight=None, k_weight=None, axes=None,
             inv_freq=(1e4 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev))
    if case["norm"]:
        s.update(q_weight=(1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt), k_weight=(1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt))
    t = torch.arange(T, dtype=torch.int32, device=dev)
    if case["axes"] == 1:
        s["positions"] = case["start"] + t
    else:  # frames of 12 rows of 20 patches
        s["positions"] = case["start"] + torch.stack([t // 240, (t // 20) % 12, t % 20][:case["axes"]])
        s["axes"] = torch.arange(half, dtype=torch.int32, device=dev) % case["axes"]
    if case["op"] == "append":
        page = case["page"]
        pages = -(-T // page) + 3
        kc, vc = _empty_cache(case, pages, dev), _empty_cache(case, pages, dev)
        order = host.permutation(pages).astype(np.int64)
        at = np.arange(T)
        slots = order[at // page] * page + at % page
        s.update(v=qkv[:, case["Hq"] + Hkv:], k_cache=kc[0], k_scale=kc[1], v_cache=vc[0], v_scale=vc[1], table=_ints(order[None].tolist(), dev),
                 cu=_ints([0, T], dev))
        slots[host.random(T) < 0.02] = -1  # padding of a fixed batch
        s["slots"] = _ints(slots.tolist(), dev)
    return s


def _prepare_chunk(case, gen, host, dev):
    dt, Hkv, D, page = DTYPES[case["dtype"]], case["Hkv"], case["D"], case["page"]
    lens = _lengths(case["B"], case["ctx"], case["spread"])
    new = [min(case["new"], n) for n in lens]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    places = host.permutation(pages)[:sum(held)].astype(np.int32)
    table = np.full((len(lens), max(held)), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = places[at:at + n]
        at += n
    wide = torch.where(torch.rand(Hkv, D, generator=gen, device=dev) < 0.02, 8.0, 1.0)  # channels of the keys that stand out
    kc, vc = _empty_cache(case, pages, dev), _empty_cache(case, pages, dev)
    step = max(1, (1 << 26) // (Hkv * page * D))
    for side, ch in ((kc, wide[:, None, :]), (vc, None)):
        for a in range(0, pages, step):
            b = min(pages, a + step)
            codes, scales = _encode(_normal((b - a, Hkv, page, D), gen, dt, ch), case["mode"])
            side[0][a:b] = codes
            if scales is not None:
                side[1][a:b] = scales
    return dict(case=case, k_cache=kc[0], k_scale=kc[1], v_cache=vc[0], v_scale=vc[1], table=torch.from_numpy(table).to(dev),
                lengths=_ints(lens, dev), cu=_ints([0, *np.cumsum(new).tolist()], dev), max_new=max(new), max_length=max(lens),
                q=_normal((sum(new), case["Hq"], D), gen, dt))


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    if case["op"] == "gemm":
        return _prepare_gemm(case, gen, dev)
    return _prepare_chunk(case, gen, host, dev) if case["op"] == "chunk" else _prepare_rows(case, gen, host, dev)


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


def _rotated(s, x, weight):
    """Rows [T, heads, D] in fp32, normed where there is a weight, the first R elements rotated."""
    case, x = s["case"], x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    pos = s["positions"] if s["axes"] is None else s["positions"][s["axes"].long()].T
    angle = (pos[:, None] if s["axes"] is None else pos).double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    R = case["R"]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["turn"] else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if case["turn"] else torch.cat([u, v], -1), x[..., R:]], -1)


def _held(s):
    """What the cache holds, as a caller can use it: its tensors, or the values of int8 codes."""
    if s["case"]["mode"] != "int8":
        return tuple(t for t in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]) if t is not None)
    t = torch.arange(s["case"]["T"], device=s["table"].device)
    return tuple(x.to(DTYPES[s["case"]["dtype"]]) for x in _gather(s, torch.zeros_like(t), t))


def _plain_rows(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    q, k = _rotated(s, s["q"], s["q_weight"]), _rotated(s, s["k"], s["k_weight"])
    if case["op"] == "rope":
        return q.to(dt), k.to(dt)
    page, mode = case["page"], case["mode"]
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][at]
    p, o = (slots // page).long(), (slots % page).long()
    for new, codes, scales in ((k[at], s["k_cache"], s["k_scale"]), (s["v"][at], s["v_cache"], s["v_scale"])):
        c, sc = _encode(new, mode)
        if mode == "e4m3":
            codes, c = codes.view(torch.uint8), c.view(torch.uint8)
        codes[p, :, o] = c.to(codes.dtype)
        if sc is not None:
            scales[p, :, o] = sc
    return (q.to(dt), *_held(s))


def _plain_chunk(s):
    """Softmax attention of the new rows, padded to [B, rows], over all positions; what a row does not see is masked."""
    case, dev = s["case"], s["q"].device
    Hq, Hkv, D, most, n = case["Hq"], case["Hkv"], case["D"], s["max_new"], s["max_length"]
    B = s["lengths"].shape[0]
    i, j = torch.arange(most, device=dev), torch.arange(n, device=dev)
    new = s["cu"][1:] - s["cu"][:-1]
    q = s["q"][(s["cu"][:-1, None] + i).clamp_(max=s["q"].shape[0] - 1)].float() * (1.0 / math.sqrt(D))
    k, v = _gather(s, torch.arange(B, device=dev)[:, None], j[None])
    last = ((s["lengths"] - new)[:, None] + i)[..., None]  # a row's own position
    seen = (j <= last) & (j < s["lengths"][:, None, None])
    if case["window"]:
        seen &= (j > last - case["window"]) | (j < case["sinks"])
    v = torch.where((j < s["lengths"][:, None])[..., None, None], v, 0.0)
    q = q.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(B, Hkv, -1, most, n)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, n), v.permute(0, 2, 1, 3).contiguous()).view(B, Hkv, -1, most, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    return o[i < new[:, None]].to(DTYPES[case["dtype"]])


def _plain(s):
    op = s["case"]["op"]
    if op == "gemm":  # (sums of products of codes pass 2^24)
        acc = torch.matmul(s["a"].double(), s["w"].double().T)
        return (acc.float() * (s["a_scale"][:, None] * s["w_scale"])).to(DTYPES[s["case"]["dtype"]])
    return _plain_chunk(s) if op == "chunk" else _plain_rows(s)


# ---- one pass --------------------------------------------------------------------------------

def _own(s):
    import flatquant_transform_quant_amd as fq

    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if case["op"] == "gemm":
        return fq.int8_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=dt)
    if case["op"] == "rope":
        return fq.qk_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                          interleaved=case["turn"], axes=s["axes"])
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside the tensors
        mode = case["dtype"] if case["mode"] == "same" else case["mode"]
        cache = s["cache"] = fq.KVCache(mode, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if case["op"] == "chunk":
        return fq.attn_chunk(s["q"], cache, s["table"], s["cu"], s["lengths"], window=case["window"], sinks=case["sinks"])
    q = fq.kv_append(cache, s["q"], s["k"], s["v"], s["slots"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                     k_weight=s["k_weight"], eps=EPS, interleaved=case["turn"], axes=s["axes"])
    if case["mode"] == "int8":
        return (q, *fq.kv_read(cache, s["table"], s["cu"], case["T"], dt))
    return (q, *_held(s))


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in fp64 --------------------------------------------------------------------

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


def _turned64(s, x, weight):
    """The rows as complex numbers, each pair turned by its angle."""
    case, x = s["case"], x.double()
    if weight is not None:
        x = weight.double() * (x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS))
    R = case["R"]
    pairs = x[..., :R].unflatten(-1, (R // 2, 2) if case["turn"] else (2, R // 2))
    z = torch.complex(*pairs.unbind(-1 if case["turn"] else -2))
    pos = s["positions"].double().reshape(-1, case["T"])
    which = torch.zeros(R // 2, dtype=torch.long, device=x.device) if s["axes"] is None else s["axes"].long()
    turn = pos.T[:, which] * s["inv_freq"].double()
    z = z * torch.polar(torch.ones_like(turn), turn)[:, None]
    return torch.cat([torch.stack([z.real, z.imag], -1 if case["turn"] else -2).flatten(-2), x[..., R:]], -1)


def _rows64(s):
    case = s["case"]
    q, k = _turned64(s, s["q"], s["q_weight"]), _turned64(s, s["k"], s["k_weight"])
    if case["op"] == "rope":
        return q, k
    page, mode, T = case["page"], case["mode"], case["T"]
    there = (s["slots"] >= 0)[:, None]
    pages = s["k_cache"].shape[0]
    values, scales = [], []
    for x in (k, s["v"].double()):
        x = x * there[..., None]
        sc = None
        if mode != "same":  # (the scale, and the quotient that is rounded to a code, are fp32 numbers by the format's definition)
            sc = (x.abs().amax(-1) / QMAX[mode]).float().double()
            y = torch.where(sc[..., None] > 0, x / sc[..., None].clamp(min=1e-300), 0.0).float().double()
            x = _nearest(y, mode) if mode == "e4m3" else y.round().clamp(-127.0, 127.0) * sc[..., None]
        if mode != "int8":  # token t of the only sequence lies in page table[0, t / page]
            def place(rows):
                full = torch.zeros(pages * page, *rows.shape[1:], dtype=torch.float64, device=rows.device)
                full[:T] = rows
                out = torch.empty_like(full).view(pages, page, *rows.shape[1:])
                out[s["table"][0].long()] = full.view(pages, page, *rows.shape[1:])
                return out.transpose(1, 2)
            x, sc = place(x), None if sc is None else place(sc)
        values.append(x)
        scales.append(sc)
    return (q, *values, *([] if mode in ("same", "int8") else scales))


def _sequence64(s, side, pages):
    """One side's values [tokens, heads, D] in the order of `pages`."""
    codes, scales, mode = s[side + "_cache"], s[side + "_scale"], s["case"]["mode"]
    codes = codes[pages] if mode == "same" else codes.view(torch.uint8)[pages]  # (indexed as bytes)
    return _values64(codes, None if scales is None else scales[pages], mode).transpose(1, 2).reshape(-1, s["case"]["Hkv"], s["case"]["D"])


def _chunk64(s):
    case, page, D = s["case"], s["case"]["page"], s["case"]["D"]
    lens, cu, Hq, Hkv = s["lengths"].tolist(), s["cu"].tolist(), case["Hq"], case["Hkv"]
    out = torch.zeros(cu[-1], Hq, D, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(lens):
        pages = s["table"][b, :-(-n // page)].long()
        k, v = (_sequence64(s, x, pages)[:n] for x in ("k", "v"))
        j = torch.arange(n, device=k.device)
        for r in range(cu[b], cu[b + 1], 2048):
            e = min(cu[b + 1], r + 2048)
            at = n - cu[b + 1] + torch.arange(r, e, device=k.device)[:, None]
            hidden = j > at
            if case["window"]:
                hidden |= (j <= at - case["window"]) & (j >= case["sinks"])
            for h in range(Hq):
                p = torch.softmax((s["q"][r:e, h].double() @ k[:, h * Hkv // Hq].T / math.sqrt(D)).masked_fill_(hidden, -math.inf), -1)
                out[r:e, h] = p @ v[:, h * Hkv // Hq]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        w = s["w"].double() * s["w_scale"].double()[:, None]
        return (s["a"].double() * s["a_scale"].double()[:, None]) @ w.T
    if case["op"] == "chunk":
        return None if case["Hq"] * case["D"] * sum(min(case["new"], n) * n for n in _lengths(case["B"], case["ctx"], case["spread"])) > 1e13 else _chunk64(s)
    return _rows64(s)
