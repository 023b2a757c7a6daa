"""GPU: attention of packed prompts where row numbers are out of order, against fp64 with the derived elementwise bound."""
import math

import pytest
import torch

import flatquant_transform_quant_amd as fq
from attn_ref import bound, softmax_attend
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
