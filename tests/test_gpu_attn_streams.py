"""GPU: memory that calls on a caller's stream allocate, while the current stream is still busy."""
import pytest
import torch

import flatquant_transform_quant_amd as fq
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def test_blocks_that_the_current_stream_still_writes():
    """Blocks of the sizes that the calls need are given back while long work and then writes to them are pending on the
    current stream: the calls on another stream, which does not wait for that work, must not be given them."""
    g = torch.Generator(device=DEV).manual_seed(0)
    B, Hq, H, D, P, width = 3, 8, 2, 128, 16, 60
    rows = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    cache = fq.empty_kv_cache(B * width, H, P, D, "int8", DEV)
    n = B * width * P
    fq.kv_write(cache, rows(n, H, D), rows(n, H, D), torch.arange(n, dtype=torch.int32, device=DEV))
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    lens = torch.full((B,), width * P, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 700, 1500, 1501], dtype=torch.int32, device=DEV)
    q, pq, pk = rows(B, Hq, D), rows(100, 4, D), rows(2000, 2, D)
    cq, ck = (torch.tensor([0, m], dtype=torch.int32, device=DEV) for m in (100, 2000))
    x, p = rows(64, 256, 256), rows(256, 256)
    codes, sc = fq.empty_outputs(64, 256, 256, "int4", DEV)

    def calls(stream):
        fq.quantize(x, p, p, codes, sc, "int4", stream=stream)
        return [*fq.kv_read(cache, table, cu, 1501, torch.bfloat16, stream=stream), fq.attn_decode(q, cache, table, lens, stream=stream),
                fq.attn_prefill(pq, pk, pk, cq, ck, stream=stream), fq.dequantize(codes, sc, "int4", 256, 256, torch.bfloat16, stream=stream)]

    want = [t.clone() for t in calls(None)]
    sizes = [fq.attn_decode_workspace_size(q, cache, table), fq.attn_prefill_workspace_size(pq, pk, cq), 512,
             *(t.numel() * t.element_size() for t in want)]
    assert sizes[0] > 0 and sizes[1] > 0
    big = rows(8192, 8192)
    side = torch.cuda.Stream()
    for r in range(3):
        say(f"[gpu] pending writes {r}")
        torch.cuda.synchronize()
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
        for _ in range(10):
            big @ big  # some 10 ms
        for b in blocks:
            b.fill_(255)
        del blocks, b
        got = calls(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want))
