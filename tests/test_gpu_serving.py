"""GPU: int8 projections, rotation with the append, and attention of new tokens over the cache as a program runs them together --
the example layer, captured runs, several host threads, memory of other streams."""
import os
import sys
import threading

import pytest
import torch

import flatquant_transform_quant_amd as fq
from gpu_util import DEV, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu

# As in the example's first test: attention outputs differ by delta of their size, and an output projection whose quantizer
# has a step of s deviations turns that into sqrt(s delta + delta^2); half as much again for a few rows.  s is 0.46 for int4
# and 0.03 for int8 (a row's largest of 1024 is about 3.3 deviations, over 7 and 127).  With a window every way reads the
# cache, whose codes depend on the token alone: what differs is bf16 rounding (0.4%) of weights and outputs.
DELTA = {"bf16": 0.004, "int8": 0.0093, "e4m3": 0.037, "int4": 0.17, "fp4": 0.17}
STEP = {4: 0.46, 8: 0.03}


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 0), (24, 3)])
@pytest.mark.parametrize("mode", list(DELTA))
def test_layer_prompt_chunks_steps_and_drafts_agree(mode, window, sinks, bits):
    import attention_layer

    delta = DELTA["bf16" if window else mode]
    most = 1.5 * (STEP[bits] * delta + delta ** 2) ** 0.5
    for drafts in (False, True):
        say(f"[gpu] layer {mode} window {window} sinks {sinks} bits {bits} drafts {drafts}")
        chunks, steps = attention_layer.run(mode, 16, 64, heads=8, kv_heads=2, counts=(70, 9, 33), steps=3, drafts=drafts, bits=bits,
                                            base=1e4, window=window, sinks=sinks)
        say(f"[gpu]   chunks {chunks:.4f} steps {steps:.4f}, at most {most:.4f}")
        assert chunks < most and steps < most


class State:
    """B sequences of `each` new tokens behind cached ones, a layer's projections, and buffers for a run without allocations."""

    def __init__(self, mode, B=3, each=5, Hq=8, H=2, D=64, P=16, width=200, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rows = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
        self.M, self.N, self.mode, self.T, self.each, self.P, self.heads = 16, 32, mode, B * each, each, P, (Hq, H, D)
        K = self.M * self.N
        self.p1, self.p2 = (torch.linalg.qr(rows(n, n).float())[0].bfloat16().contiguous() for n in (self.M, self.N))
        weight = lambda o: (torch.randint(-127, 128, (o, K), generator=g, device=DEV).to(torch.int8),  # noqa: E731
                            torch.rand(o, generator=g, device=DEV) * 1e-3 + 1e-4)
        self.qkv, self.proj = weight((Hq + 2 * H) * D), weight(K)
        self.norms = rows(2, D)
        self.freq = 1e4 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float32) / D)
        self.cache = fq.empty_kv_cache(B * width, H, P, D, mode, DEV)
        self.table = torch.randperm(B * width, device=DEV, generator=g).to(torch.int32).view(B, width)
        n = B * width * P
        fq.kv_write(self.cache, rows(n, H, D), rows(n, H, D), torch.arange(n, dtype=torch.int32, device=DEV))
        self.x = rows(self.T, self.M, self.N)
        self.cu = torch.arange(B + 1, dtype=torch.int32, device=DEV) * each
        self.lens, self.at, self.slots = (torch.zeros(m, dtype=torch.int32, device=DEV) for m in (B, self.T, self.T))
        self.ws = torch.empty(self.need(), dtype=torch.uint8, device=DEV)

    def need(self):
        Hq, _, D = self.heads
        q = torch.empty(self.T, Hq, D, dtype=torch.bfloat16, device=DEV)
        return fq.attn_chunk_workspace_size(q, self.cache, self.table, self.cu, 2000, 4)

    def place(self, lens):
        """The new tokens are the last of the sequences' `lens` ones."""
        t = torch.tensor(lens)[:, None] - self.each + torch.arange(self.each)[None]
        pages = self.table.cpu().gather(1, (t // self.P).long())
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.at.copy_(t.reshape(-1).int())
        self.slots.copy_((pages * self.P + t % self.P).reshape(-1).int())

    def linear(self, x, w):
        codes, sc = fq.empty_outputs(self.T, self.M, self.N, "int8", DEV)
        fq.quantize(x.view(self.T, self.M, self.N), self.p1, self.p2, codes, sc, "int8")
        return fq.int8_gemm(codes.view(self.T, -1), sc, *w)

    def run(self, ws=None):
        Hq, H, D = self.heads
        y = self.linear(self.x, self.qkv).view(self.T, Hq + 2 * H, D)
        q = fq.kv_append(self.cache, y[:, :Hq], y[:, Hq:Hq + H], y[:, Hq + H:], self.slots, self.at, self.freq, *self.norms)
        o = fq.attn_chunk(q, self.cache, self.table, self.cu, self.lens, 2000, 4, workspace=ws)
        return self.linear(o, self.proj)


@pytest.mark.parametrize("mode", ["bf16", "int8", "fp4"])
def test_a_captured_run_replays(mode):
    """Projection, append, attention and projection in a graph, twice with workspaces of their own: every replay equals the
    eager run on the inputs of the moment."""
    say(f"[gpu] captured run {mode}")
    s = State(mode)
    s.place([5, 100, 3200])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(s.ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs, spaces = [], [], [s.ws, torch.empty_like(s.ws)]
    for ws in spaces:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(s.run(ws))
    for r, lens in enumerate(([5, 100, 3200], [6, 2017, 33], [3199, 64, 5], [2001, 3200, 1999])):
        s.place(lens)
        s.x.copy_(torch.randn(s.x.shape, device=DEV))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = s.run()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], want), r


def test_several_host_threads():
    """Threads, each on its own stream with its own cache: the same results as alone."""
    jobs = [State(m, seed=i) for i, m in enumerate(("int8", "fp4", "bf16", "int4"))]
    want = []
    for i, s in enumerate(jobs):
        s.place([5, 100 + i, 3190])
        want.append(s.run())
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out = jobs[i].run()
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(out, want[i]):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad, bad


def test_blocks_that_the_current_stream_still_writes():
    """Results and workspaces of calls on another stream never lie in blocks that the current stream has work on."""
    s = State("int8", B=4, each=16, width=220)
    s.place([16, 300, 2700, 3500])
    Hq, H, D = s.heads
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k = (torch.randn(s.T, h, D, generator=g, device=DEV).bfloat16() for h in (Hq, H))
    codes, sc = fq.empty_outputs(s.T, s.M, s.N, "int8", DEV)
    fq.quantize(s.x, s.p1, s.p2, codes, sc, "int8")

    def calls(stream):
        return [*fq.qk_rope(q, k, s.at, s.freq, *s.norms, stream=stream),
                fq.kv_append(s.cache, q, k, k, s.slots, s.at, s.freq, *s.norms, stream=stream),
                fq.attn_chunk(q, s.cache, s.table, s.cu, s.lens, stream=stream), fq.int8_gemm(codes.view(s.T, -1), sc, *s.qkv, stream=stream)]

    want = [t.clone() for t in calls(None)]
    sizes = [fq.attn_chunk_workspace_size(q, s.cache, s.table, s.cu), *(t.numel() * t.element_size() for t in want)]
    assert sizes[0] > 0
    big = torch.randn(8192, 8192, device=DEV).bfloat16()
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
