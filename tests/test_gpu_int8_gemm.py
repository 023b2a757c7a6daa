"""GPU: the int8 consumer GEMM.  The integer sums are exact and the scaling is a fixed sequence of fp32 operations, so every
result is one defined value, compared bit for bit with sums in 64-bit integers."""
import numpy as np
import pytest
import torch

import flatquant_transform_quant_amd as fq
import synth
from gpu_util import DEV, run_lib, say, to_dev

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def want_of(a, sa, w, sw, dt):
    """fl32(acc) * fl32(sa sw) in numpy (fp64 products of codes and their sums are exact below 2^53)."""
    acc = (a.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)
    with np.errstate(over="ignore"):
        return torch.from_numpy(acc.astype(np.float32) * (sa[:, None] * sw[None])).to(dt)


def operands(T, O, H, seed, spread=4.0):
    g = np.random.default_rng(seed)
    side = lambda n: (g.integers(-128, 128, (n, H), dtype=np.int8), np.exp(g.uniform(-spread, spread, n)).astype(np.float32))  # noqa: E731
    return (*side(T), *side(O))


def check(T, O, H, dt, seed):
    a, sa, w, sw = operands(T, O, H, seed)
    say(f"[gpu] int8_gemm T={T} O={O} H={H} {dt}")
    out = torch.full((T + 1, O), 7.0, dtype=dt, device=DEV)
    got = fq.int8_gemm(*(torch.from_numpy(x).to(DEV) for x in (a, sa, w, sw)), out=out[:T])
    want = want_of(a, sa, w, sw, dt)
    bits = torch.int32 if dt == torch.float32 else torch.int16
    assert torch.equal(got.cpu().view(bits), want.view(bits)) and (out[T] == 7.0).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,O,H", [(1, 1, 16), (1, 16, 128), (3, 5, 48), (16, 33, 1040), (17, 64, 2048), (32, 130, 4112), (33, 31, 8192), (64, 257, 160),
                                   (65, 1, 16), (65, 128, 256), (127, 129, 1024), (130, 300, 80), (300, 200, 4112), (129, 2, 8208)])
def test_sizes(T, O, H, dt):
    check(T, O, H, dt, T + O + H)


@pytest.mark.parametrize("T,O,H", [(4096, 4096, 144), (4097, 4100, 272), (300, 33000, 64), (33000, 300, 16)])
def test_large(T, O, H):
    check(T, O, H, torch.bfloat16, 1)


@pytest.mark.parametrize("T,O,H", [(300, 9001, 80), (300, 9000, 400), (257, 10900, 1040), (1000, 5000, 144), (1001, 4999, 1168), (200, 60000, 272)])
def test_middle_tiles(T, O, H):
    """Tiles of 128 by 128 and by 256, walks shorter and longer than their buffers."""
    check(T, O, H, torch.bfloat16, 2)


@pytest.mark.parametrize("T", [1, 20, 50, 100, 2000])
def test_rows_do_not_depend_on_their_number(T):
    """The same row gives the same bits whatever kernel the number of rows chooses."""
    a, sa, w, sw = (torch.from_numpy(x).to(DEV) for x in operands(2000, 2050, 528, 3))
    full = fq.int8_gemm(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.equal(fq.int8_gemm(a[:T].contiguous(), sa[:T].contiguous(), w, sw, out_dtype=torch.float32), full[:T])


@pytest.mark.parametrize("T", [2, 40, 100])
def test_extreme_codes_and_scales(T):
    """Every code -128 at the largest H: the largest sum, below 2^31; scales that overflow, are zero, infinite or NaN."""
    H = 2 ** 17 - 16
    a = torch.full((T, H), -128, dtype=torch.int8, device=DEV)
    w = torch.full((5, H), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    w[2] = 0
    sa = torch.ones(T, device=DEV)
    sa[1] = 3e38
    sw = torch.tensor([1.0, 1.0, 1.0, 0.0, float("nan")], device=DEV)
    got = fq.int8_gemm(a, sa, w, sw, out_dtype=torch.float32).cpu()
    first = torch.tensor([16384.0 * H, -16256.0 * H, 0.0, 0.0])
    assert torch.equal(got[0, :4], first) and torch.isnan(got[:, 4]).all()
    assert got[1, 0] == float("inf") and got[1, 1] == -float("inf") and (got[:, 2:4] == 0).all()


@pytest.mark.parametrize("T", [1, 70])
def test_outputs_at_odd_places(T):
    """A C whose rows are not whole vectors, at an address that is not aligned to one."""
    a, sa, w, sw = operands(T, 7, 96, 5)
    dev = [torch.from_numpy(x).to(DEV) for x in (a, sa, w, sw)]
    for dt in TYPES:
        flat = torch.full((T * 7 + 2,), 9.0, dtype=dt, device=DEV)
        fq.int8_gemm(*dev, out=flat[1:-1].view(T, 7))
        assert torch.equal(flat[1:-1].view(T, 7).cpu(), want_of(a, sa, w, sw, dt)) and flat[0] == 9.0 and flat[-1] == 9.0
        # O a multiple of four, C not aligned
        got = torch.full((T * 4 + 1,), 9.0, dtype=dt, device=DEV)
        fq.int8_gemm(dev[0], dev[1], dev[2][:4], dev[3][:4], out=got[1:].view(T, 4))
        assert torch.equal(got[1:].view(T, 4).cpu(), want_of(a, sa, w[:4], sw[:4], dt))


def test_consumes_the_quantizer_output():
    """A = the per-token int8 output of the quantizer (64 x 64 slices as tokens) with its scales."""
    w_ = synth.WORKLOADS["c2i8"]
    K, H = 96, w_.M * w_.N
    x, p1, p2 = synth.make_inputs(w_, 0, K)
    out, sc = run_lib(to_dev(x, w_.dtype), to_dev(p1, w_.dtype), to_dev(p2, w_.dtype), w_.mode, w_.clip_ratio, w_.dst_type_max)
    _, _, w, sw = operands(1, 160, H, 7)
    got = fq.int8_gemm(out.view(K, H), sc, torch.from_numpy(w).to(DEV), torch.from_numpy(sw).to(DEV), out_dtype=torch.float32)
    assert torch.equal(got.cpu(), want_of(out.view(K, H).cpu().numpy(), sc.cpu().numpy(), w, sw, torch.float32))


def test_nothing_to_do():
    one, f = torch.zeros(3, 32, dtype=torch.int8, device=DEV), torch.zeros(3, device=DEV)
    assert fq.int8_gemm(one[:0], f[:0], one, f).shape == (0, 3)
    assert fq.int8_gemm(one, f, one[:0], f[:0]).shape == (3, 0)


def test_operands_past_32_bits():
    """Rows of A, rows of W and results whose places lie past 2^31 bytes and elements."""
    H = 65536
    a = torch.zeros(70000, H, dtype=torch.int8, device=DEV)  # 4.6 GB
    a[:, 5] = 1
    a[-1] = 3
    sa, w, sw = torch.ones(70000, device=DEV), torch.ones(3, H, dtype=torch.int8, device=DEV), torch.ones(3, device=DEV)
    say("[gpu] int8_gemm past 4 GB")
    got = fq.int8_gemm(a, sa, w, sw, out_dtype=torch.float32)
    assert (got[:-1] == 1).all() and (got[-1] == 3.0 * H).all()
    got = fq.int8_gemm(w, sw, a, sa, out_dtype=torch.float32)
    assert (got[:, :-1] == 1).all() and (got[:, -1] == 3.0 * H).all()
    del a, got
    n = 50000
    a, s = torch.ones(n, 16, dtype=torch.int8, device=DEV), torch.arange(n, dtype=torch.float32, device=DEV)
    got = fq.int8_gemm(a, s, a, torch.ones(n, device=DEV))  # 2.5 10^9 elements
    assert torch.equal(got[-3:].float(), (16.0 * s[-3:, None]).bfloat16().float().expand(3, n))


def test_captured_and_on_another_stream():
    for T in (5, 100):
        a, sa, w, sw = (torch.from_numpy(x).to(DEV) for x in operands(T, 300, 1040, 9))
        fq.int8_gemm(a, sa, w, sw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fq.int8_gemm(a, sa, w, sw)
        for i in range(3):
            a.add_(1), sa.mul_(1.5)
            want = fq.int8_gemm(a, sa, w, sw)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = fq.int8_gemm(a, sa, w, sw, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
