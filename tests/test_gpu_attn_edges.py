"""GPU: attention at the edges of its inputs' ranges, against fp64 or known results."""
import math

import pytest
import torch

import flatquant_transform_quant_amd as fq
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
