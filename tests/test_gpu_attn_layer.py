"""GPU: the cache and attention calls as a program runs them -- the example layer, captured steps, other
streams, several host threads."""
import os
import sys
import threading

import pytest
import torch

import flatquant_transform_quant_amd as fq
from gpu_util import DEV, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


# The layer's last rows, with the cache's rounding in them, against the whole prompt's (whose attention reads the keys and
# values as they were projected).  The attention outputs differ by delta of their size: a format's relative error of a
# value (int8, int4: the step max / 127, / 7 over sqrt(12), max about 2.9 of a deviation; E4M3 2.6%, E2M1 12%), times
# sqrt(2) for the keys' part in the weights; bf16 0.4% for roundings.  The output projection's int4 quantizer (step 0.46 of
# a deviation) turns that into sqrt(0.46 delta + delta^2) by the codes that flip; half as much again for a few rows.
DELTA = {"bf16": 0.004, "int8": 0.0093, "e4m3": 0.037, "int4": 0.17, "fp4": 0.17}


@pytest.mark.parametrize("mode", list(DELTA))
def test_layer_prompt_chunks_and_steps_agree(mode):
    import attention_layer

    most = 1.5 * (0.46 * DELTA[mode] + DELTA[mode] ** 2) ** 0.5
    say(f"[gpu] layer {mode}")
    chunks, steps = attention_layer.run(mode, 16, 64, heads=8, kv_heads=2, counts=(70, 9, 33), steps=3)
    say(f"[gpu]   chunks {chunks:.4f} steps {steps:.4f}")
    assert chunks < most and steps < most


def _state(mode="int8", B=5, Hq=8, H=2, D=128, P=16, width=40, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = fq.empty_kv_cache(B * width, H, P, D, mode, DEV)
    table = torch.randperm(B * width, device=DEV, generator=g).to(torch.int32).view(B, width)
    n = width * P
    rows = lambda t, h: torch.randn(t, h, D, generator=g, device=DEV).bfloat16()  # noqa: E731
    fq.kv_write(cache, rows(B * n, H), rows(B * n, H), torch.arange(B * n, dtype=torch.int32, device=DEV))
    return cache, table, rows(B, Hq), rows(B, H), rows(B, H)


def _step(cache, table, q, k, v, slots, lens, ws, out):
    fq.kv_write(cache, k, v, slots)
    fq.attn_decode(q, cache, table, lens, workspace=ws, out=out)


@pytest.mark.parametrize("mode", ["bf16", "int4", "fp4"])
def test_a_captured_step_replays(mode):
    """A decode step (write, attention, join) in a graph: every replay equals the eager step on the inputs of the moment,
    with lengths, slots and pages read on the device."""
    say(f"[gpu] graph {mode}")
    cache, table, q, k, v = _state(mode)
    B, P = q.shape[0], cache.page_size
    lens = torch.tensor([1, 0, 600, 33, 129], dtype=torch.int32, device=DEV)
    slots = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    ws = torch.empty(fq.attn_decode_workspace_size(q, cache, table), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(cache, table, q, k, v, slots, lens, ws, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(cache, table, q, k, v, slots, lens, ws, out)
    for r in range(4):
        lens.copy_((lens + 97 * r) % 640)
        slots.copy_(torch.where(lens > 0, table.gather(1, ((lens - 1).clamp(min=0) // P).long()[:, None])[:, 0] * P + (lens - 1) % P, -1))
        q.copy_(torch.randn(q.shape, device=DEV))
        k.copy_(torch.randn(k.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = torch.empty_like(out)
        _step(cache, table, q, k, v, slots, lens, None, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want), r


def test_other_streams_and_freed_temporaries():
    """Calls on a side stream whose workspaces and outputs come from the current stream's allocator; blocks freed right away
    are taken again at once by work on the current stream."""
    cache, table, q, k, v = _state()
    lens = torch.full((q.shape[0],), 640, dtype=torch.int32, device=DEV)
    want = fq.attn_decode(q, cache, table, lens)
    cu = torch.tensor([0, 2000], dtype=torch.int32, device=DEV)
    cq = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    pq, pk, pv = (torch.randn(n, h, 128, device=DEV).bfloat16() for n, h in ((100, 4), (2000, 2), (2000, 2)))
    want_p = fq.attn_prefill(pq, pk, pv, cq, cu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append((fq.attn_decode(q, cache, table, lens, stream=side), fq.attn_prefill(pq, pk, pv, cq, cu, stream=side)))
        junk = [torch.full((4 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(6)]
        del junk
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want) and torch.equal(b, want_p)


def test_several_host_threads():
    """Threads, each on its own stream, at different calls: the same results as alone."""
    jobs, want = [], []
    for i, mode in enumerate(("int8", "fp4", "bf16", "e4m3")):
        cache, table, q, k, v = _state(mode, seed=i)
        lens = torch.tensor([640, 3, 400, 17, 0], dtype=torch.int32, device=DEV)
        jobs.append((cache, table, q, lens))
        want.append(fq.attn_decode(q, cache, table, lens))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out = fq.attn_decode(jobs[i][2], jobs[i][0], jobs[i][1], jobs[i][3])
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(out, want[i]):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad, bad
