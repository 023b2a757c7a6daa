"""An attention layer served in low bits: int4 projections (transform + quantize, int4 GEMM), a paged
low-bit key-value cache, prompts in packed chunks and single tokens in batches.

    python examples/attention_layer.py [--mode int8] [--hidden 4096]

The activations go through random orthogonal transforms P1, P2 (Kronecker factors of a rotation of
the hidden dimension), the weights through their inverse once, so that x W^T is unchanged but
for the quantization.  No checkpoint is loaded: weights are random.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import flatquant_transform_quant_amd as fq  # noqa: E402


class Int4Linear:
    """y = W x with x [T, M*N] transformed and quantized per token, W int4 per output channel."""

    def __init__(self, W, M: int, N: int, gen):
        dev = W.device
        orth = lambda n: torch.linalg.qr(torch.randn(n, n, generator=gen, device=dev))[0].to(torch.bfloat16).contiguous()  # noqa: E731
        self.M, self.N, self.p1, self.p2 = M, N, orth(M), orth(N)
        # P1 X P2 of the row x as a matrix is (P1 kron P2^T) x; its inverse goes into W
        R = torch.kron(self.p1.float(), self.p2.float().T.contiguous())
        Wr = torch.linalg.solve(R.T.contiguous(), W.T.contiguous()).T.contiguous()
        scale = Wr.abs().amax(1) / 7.0
        q = (Wr / scale[:, None]).round().clamp(-8, 7).to(torch.int8).view(torch.uint8) & 15
        self.codes, self.scale = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scale.contiguous()

    def __call__(self, x):
        T = x.shape[0]
        out, sc = fq.empty_outputs(T, self.M, self.N, "int4", x.device)
        fq.quantize(x.view(T, self.M, self.N), self.p1, self.p2, out, sc, "int4")
        return fq.int4_gemm(out.view(T, -1), sc, self.codes, self.scale, self.M * self.N)


class AttentionLayer:
    def __init__(self, M: int, N: int, heads: int, kv_heads: int, mode: str, pages: int, page_size: int, max_batch: int,
                 max_pages: int, device="cuda", seed: int = 0):
        hidden, self.Hq, self.H, self.D = M * N, heads, kv_heads, M * N // heads
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda o: torch.randn(o, hidden, generator=gen, device=device) / hidden ** 0.5  # noqa: E731
        self.qkv = Int4Linear(rand((heads + 2 * kv_heads) * self.D), M, N, gen)
        self.out = Int4Linear(rand(hidden), M, N, gen)
        self.cache = fq.empty_kv_cache(pages, kv_heads, page_size, self.D, mode, device)
        # the scheduler's side: which pages each sequence of the batch holds, and how many tokens
        self.free = list(range(pages))[::-1]
        self.table = torch.full((max_batch, max_pages), -1, dtype=torch.int32)
        self.lengths = [0] * max_batch
        self.P, self.device = page_size, device

    def _slots(self, seqs, counts):
        """Slots of the next counts[i] tokens of sequence seqs[i], with pages taken as needed."""
        slots = []
        for s, n in zip(seqs, counts):
            for t in range(self.lengths[s], self.lengths[s] + n):
                if t % self.P == 0:
                    self.table[s, t // self.P] = self.free.pop()
                slots.append(int(self.table[s, t // self.P]) * self.P + t % self.P)
            self.lengths[s] += n
        return torch.tensor(slots, dtype=torch.int32, device=self.device)

    def _heads(self, x):
        y = self.qkv(x).view(x.shape[0], -1, self.D)
        return y[:, :self.Hq], y[:, self.Hq:self.Hq + self.H], y[:, self.Hq + self.H:]  # strided views

    def _cu(self, counts):
        return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(self.device)

    def prompt(self, x, seqs, counts):
        """Rows of several sequences' next chunks, packed: x [sum(counts), hidden]."""
        q, k, v = self._heads(x)
        behind = any(self.lengths[s] for s in seqs)
        fq.kv_write(self.cache, k, v, self._slots(seqs, counts))
        cu = cu_k = self._cu(counts)
        if behind:  # the chunk also attends to what is in the cache already
            lens = [self.lengths[s] for s in seqs]
            cu_k = self._cu(lens)
            k, v = fq.kv_read(self.cache, self.table[seqs].to(self.device), cu_k, sum(lens), x.dtype)
        o = fq.attn_prefill(q, k, v, cu, cu_k)
        return self.out(o.view(x.shape[0], -1))

    def step(self, x, seqs):
        """One new token of each sequence: x [len(seqs), hidden]."""
        q, k, v = self._heads(x)
        fq.kv_write(self.cache, k, v, self._slots(seqs, [1] * len(seqs)))
        lens = torch.tensor([self.lengths[s] for s in seqs], dtype=torch.int32, device=self.device)
        o = fq.attn_decode(q, self.cache, self.table[seqs].to(self.device), lens)
        return self.out(o.view(x.shape[0], -1))


def run(mode: str, M: int = 64, N: int = 64, heads: int = 32, kv_heads: int = 8, counts=(300, 41, 17), steps: int = 4, page_size: int = 16):
    """The same tokens three ways -- as one prompt, as two chunks, and a prompt followed by single steps -- and the largest
    relative difference between the ways' last rows."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    need = sum(-(-(n + steps) // page_size) for n in counts) + len(counts)
    make = lambda: AttentionLayer(M, N, heads, kv_heads, mode, need, page_size, len(counts), need)  # noqa: E731
    xs = [torch.randn(n + steps, M * N, generator=gen, device="cuda").to(torch.bfloat16) for n in counts]
    seqs, total = list(range(len(counts))), [n + steps for n in counts]
    ends = torch.tensor(total).cumsum(0) - 1
    whole = make().prompt(torch.cat(xs), seqs, total)[ends].float()
    layer = make()
    half = [n // 2 for n in total]
    layer.prompt(torch.cat([x[:h] for x, h in zip(xs, half)]), seqs, half)
    rest = [n - h for n, h in zip(total, half)]
    chunked = layer.prompt(torch.cat([x[h:] for x, h in zip(xs, half)]), seqs, rest)[torch.tensor(rest).cumsum(0) - 1].float()
    layer = make()
    layer.prompt(torch.cat([x[:n] for x, n in zip(xs, counts)]), seqs, list(counts))
    for t in range(steps):
        stepped = layer.step(torch.stack([x[n + t] for x, n in zip(xs, counts)]), seqs).float()
    off = lambda y: ((y - whole).norm() / whole.norm()).item()  # noqa: E731
    return off(chunked), off(stepped)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--mode", default="int8", choices=fq.KV_MODES)
    ap.add_argument("--hidden", type=int, default=4096, choices=(4096, 8192))
    a = ap.parse_args()
    c, s = run(a.mode, 64, a.hidden // 64, heads=a.hidden // 128)
    print(f"{a.mode} cache, hidden {a.hidden}: relative difference from the whole prompt: chunks {c:.4f}, single steps {s:.4f}")
