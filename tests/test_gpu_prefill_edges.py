"""GPU: attention of packed prompts where row numbers are out of order or scores are large, against fp64 with the derived elementwise bound."""
import math

import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import TDT, U, bound, softmax_attend
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("causal", [True, False])
def test_row_numbers_far_below_zero(causal):
    """cu_q and cu_k that do not ascend, down to the smallest int32: a sequence has no rows (or no keys) then, and those of the sequences
    beside it are right."""
    g = torch.Generator().manual_seed(40)
    r, n, D = 40, 300, 64
    q, k, v = (torch.randn(m, h, D, generator=g).bfloat16() for m, h in ((r, 4), (n, 2), (n, 2)))
    want, _, absv, top, vmax = softmax_attend(q.double(), k.double(), v.double(), torch.arange(n - r, n) + 1 if causal else torch.full((r,), n), 1 / math.sqrt(D))
    tol = bound(want, absv, top, vmax, n, D, "bf16", "bf16")
    for low in (-1, -2 ** 31, -2 ** 31 + 39):
        for cq, ck in (((0, r, low, low), (0, n, low, low)), ((r, low, r), (n, low, n)), ((0, r, r), (0, n, low))):
            say(f"[gpu] cu_q {cq} cu_k {ck} causal {causal}")
            out = torch.full((r, 4, D), 7.0, dtype=torch.bfloat16, device=DEV)
            fq.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), _i32(*cq), _i32(*ck), causal, out=out)
            assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1e3, 1e7, -1e9, 1e15, 1e30])
def test_scores_of_any_size(dt, D, scale):
    """Scores far past what fp32 tells apart by less than 1 still give means of the values that are seen, and the value of the
    key that stands out where one does by more than the scores' own error, (D + 8) 2^-24 of their terms."""
    for r, n in ((150, 400), (3, 5000)):  # (the second in parts)
        say(f"[gpu] scores {dt} D={D} scale={scale} rows={r}")
        g = torch.Generator().manual_seed(41)
        q, k, v = (torch.randn(m, h, D, generator=g).to(TDT[dt]) for m, h in ((r, 2), (n, 1), (n, 1)))
        got = fq.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), _i32(0, r), _i32(0, n), True, scale).cpu().double()
        kk, vv = k[:, 0].double(), v[:, 0].double()
        seen = torch.arange(n)[None] <= torch.arange(n - r, n)[:, None]
        s = (torch.einsum("ihd,jd->ihj", q.double(), kk) * scale).masked_fill(~seen[:, None], -math.inf)
        off = torch.einsum("ihd,jd->ihj", q.double().abs(), kk.abs()).amax(-1) * abs(scale) * (D + 8) * 2.0 ** -24
        top = s.topk(2, -1)
        least, most = vv.amin(0), vv.amax(0)
        assert torch.isfinite(got).all()
        assert (got >= least - 3 * U[dt] * least.abs()).all() and (got <= most + 3 * U[dt] * most.abs()).all()
        clear = top.values[..., 0] - top.values[..., 1] > 2 * off + 60
        assert clear.any()
        one = vv[top.indices[..., 0]]
        assert ((got - one).abs() <= 3 * U[dt] * one.abs() + 2.0 ** -24)[clear].all()
