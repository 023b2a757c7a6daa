"""Plain references of the cache and attention operators (CPU; fp64 for attention, IEEE fp32 and
explicit tables for the codes), and the error bounds their tests use."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}
TDT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # unit roundoff
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([math.ldexp(c & 7, -9) if c < 8 else math.ldexp(8 + (c & 7), (c >> 3) - 10) for c in range(127)])


def nearest_code(mags, y):
    """Index of the magnitude nearest |y|, ties to the even index."""
    a = np.abs(y.astype(np.float64))
    mid = (mags[1:] + mags[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(lo % 2 == 0, lo, hi).astype(np.int64)


def encode(x: torch.Tensor, mode: str, clip=1.0, dmax=0.0):
    """Codes (one per byte, int64) and scales (fp32, or e8m0 bytes padded to a whole number of 64s) of rows [..., D]."""
    x = x.float().numpy()
    D = x.shape[-1]
    if mode == "fp4":
        g = x.reshape(*x.shape[:-1], D // 32, 32)
        with np.errstate(all="ignore"):
            top = np.max(np.abs(g), -1)  # NaN propagates
            if dmax == 0.0:
                e8 = np.clip(np.frexp(np.where(np.isfinite(top), top, 1.0))[1].astype(np.int64) - 1 - 2 + 127, 0, 254)
                e8 = np.where(top < 2.0 ** -126, 0, e8)
            else:
                s = (top / np.float32(dmax)).astype(np.float32).view(np.uint32).astype(np.int64)
                e8 = s >> 23
                e8 = e8 + ((e8 >= 1) & (e8 < 254) & ((s & 0x7FFFFF) != 0))
            ok = np.isfinite(top)
            y = np.ldexp(g.astype(np.float64), (127 - np.where(ok, e8, 127))[..., None])
            code = nearest_code(E2M1, np.where(ok[..., None], y, 0.0)) | (np.signbit(g).astype(np.int64) << 3)
        code = np.where(ok[..., None], code, 0).reshape(x.shape)
        e8 = np.where(ok, e8, 255)
        pad = 2 * (-(-D // 64)) - D // 32
        e8 = np.concatenate([e8, np.zeros((*e8.shape[:-1], pad), np.int64)], -1)
        return code, e8
    d = np.float32(QMAX[mode] / clip)
    with np.errstate(all="ignore"):
        top = np.max(np.abs(x), -1)
        scale = (top / d).astype(np.float32)
        ok = np.isfinite(scale) & (scale > 0)
        q = np.where(ok[..., None], x / np.where(ok, scale, 1.0)[..., None].astype(np.float32), np.float32(0.0)).astype(np.float32)
    if mode == "e4m3":
        q = np.clip(q, -448.0, 448.0)
        code = nearest_code(E4M3, q) | (np.signbit(q).astype(np.int64) << 7)
    else:
        lo, hi = (-127, 127) if mode == "int8" else (-8, 7)
        code = np.clip(np.rint(q.astype(np.float64)), lo, hi).astype(np.int64) & (255 if mode == "int8" else 15)
    return code, scale


def values(code, scale, mode):
    """fp64 array of the fp32 values of codes and scales (code * scale, rounded once to fp32)."""
    if mode == "fp4":
        v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
        g = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
        e8 = scale[..., :g.shape[-2]]
        with np.errstate(all="ignore"):
            out = np.where((e8 == 255)[..., None], np.nan, np.ldexp(g, (e8 - 127)[..., None]))
        return out.reshape(v.shape)
    if mode == "int8":
        q = np.where(code >= 128, code - 256, code).astype(np.float32)
    elif mode == "int4":
        q = np.where(code >= 8, code - 16, code).astype(np.float32)
    else:
        q = (np.where(code >= 128, -1.0, 1.0) * np.append(E4M3, np.nan)[code & 127]).astype(np.float32)
    with np.errstate(all="ignore"):
        return (q * scale[..., None].astype(np.float32)).astype(np.float64)


def pack(code, mode):
    """Bytes as the cache stores them."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8) if mode in ("int4", "fp4") else code.astype(np.uint8)


def unpack(raw, mode):
    raw = raw.astype(np.int64)
    return np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], -1) if mode in ("int4", "fp4") else raw


def softmax_attend(q, k, v, n_visible, scale):
    """One sequence in fp64: q [Lq, Hq, D], k, v [Lk, Hkv, D]; row i sees keys 0 .. n_visible[i]-1.  Returns out, lse,
    sum p |v|, and the largest scale * sum |q||k| of each row (for the bounds)."""
    Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[:2]
    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    mass = torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()) * abs(scale)
    hid = torch.arange(Lk)[None] >= n_visible[:, None]
    s.masked_fill_(hid, -math.inf)
    mass.masked_fill_(hid, 0.0)
    lse = torch.logsumexp(s, -1) if Lk else torch.full((Hq, Lq), -math.inf, dtype=torch.float64)
    p = torch.where(hid, 0.0, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]))
    vz = torch.where(hid.all(0)[:, None, None], 0.0, vv) if Lk else vv  # keys no row sees
    out = torch.einsum("hij,jhd->ihd", p, vz)
    absv = torch.einsum("hij,jhd->ihd", p, vz.abs())
    top = mass.amax(-1).T if Lk else torch.zeros(Lq, Hq, dtype=torch.float64)
    vmax = vz.abs().amax(0) if Lk else torch.zeros(Hq, D, dtype=torch.float64)
    return out, lse.T, absv, top, vmax


def bound(out, absv, top, vmax, n, D, dt, p_dt):
    """Elementwise bound of an output's error.  The output's rounding: u |out|.  A weight p = exp(s) is off by the error
    of its score -- fp32 products and sums of D terms, the scale, the base-2 logarithm's factor: (D + 8) 2^-24 of
    scale * sum |q||k| -- and by exp's and the sums' own few ulp, and is rounded to p_dt before the second product: u_p.
    Numerator and denominator both carry the score's part: factor 2.  Weights below 2^-14 of the largest are f16
    subnormals, 2^-25 off each (and 2^-17 of a weight's maximum where the maximum runs up to 2^8 behind)."""
    ds = (D + 8) * 2.0 ** -24 * top[..., None]
    rel = U[p_dt] + 2.0 * ds + (16 + math.sqrt(max(n, 1))) * 2.0 ** -23
    tiny = n * 2.0 ** -25 * vmax if p_dt == "f16" else 0.0
    floor = 2.0 ** -25 if dt == "f16" else 0.0  # an output in f16's subnormal range
    return U[dt] * out.abs() + rel * absv * (1 + U[dt]) + tiny + floor
