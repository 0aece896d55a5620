"""An attention layer between two W4A4 linears over an 8-bit key/value cache.

    x --W4A4--> q, k, v;  k, v --> cache;  q, cache --attention--> o;  o --W4A4--> y

Weights are random and packed once; every step's projections, cache write and
attention run on the current stream without a host synchronisation.  Run as a
program, it takes two prompts in one call and then a few tokens of both:

    python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_block_amax_amd as fp4  # noqa: E402


class Sequences:
    """The cache's pages and the sequences that hold them (host bookkeeping)."""

    def __init__(self, pages, kv_heads, block, head_dim, device):
        self.cache = fp4.new_kv_cache(pages, kv_heads, block, head_dim, device)
        self.block, self.device = block, device
        self.free, self.held, self.lengths = list(range(pages)), [], []

    def extend(self, new):
        """Room for new[s] more tokens of each sequence (new sequences at the
        end); returns the batch: cu_tokens, lengths, table."""
        while len(self.lengths) < len(new):
            self.lengths.append(0)
            self.held.append([])
        cu = [0]
        for s, n in enumerate(new):
            cu.append(cu[-1] + n)
            self.lengths[s] += n
            while len(self.held[s]) * self.block < self.lengths[s]:
                self.held[s].append(self.free.pop())
        width = max(len(h) for h in self.held)
        table = [h + [0] * (width - len(h)) for h in self.held]
        return tuple(torch.tensor(a, dtype=torch.int32).to(self.device, non_blocking=True)
                     for a in (cu, self.lengths, table))


class AttentionLayer:
    """hidden and heads * head_dim are multiples of 2048 (the packed GEMM's K)."""

    def __init__(self, hidden, heads, kv_heads, head_dim, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):  # [n, k], packed for the GEMM
            w = torch.randn(n, k, generator=g, device=device) * k ** -0.5
            return fp4.pack_mxfp4_operand(*fp4.quantize_mxfp4(w.bfloat16()))

        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, head_dim
        self.qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, heads * head_dim)

    def project(self, x):
        """q, k and v of x [tokens, hidden]: slices of one projection's rows."""
        all_heads = self.heads + 2 * self.kv_heads
        y, _ = fp4.linear_mxfp4_packed(x, self.qkv, all_heads * self.dim, check=False)
        y = y.view(-1, all_heads, self.dim)
        return y[:, :self.heads], y[:, self.heads:-self.kv_heads], y[:, -self.kv_heads:]

    def attend(self, x, cache, batch):
        q, k, v = self.project(x)
        fp4.kv_cache_write(cache, k, v, *batch, check=False)
        return fp4.kv_attention(q, cache, *batch, check=False)

    def __call__(self, x, cache, batch):
        o = self.attend(x, cache, batch)
        return fp4.linear_mxfp4_packed(o.view(x.shape[0], -1), self.out, self.hidden,
                                       check=False)[0]


def main():
    device = torch.device("cuda")
    layer = AttentionLayer(2048, heads=16, kv_heads=2, head_dim=128, device=device)
    seqs = Sequences(pages=64, kv_heads=2, block=64, head_dim=128, device=device)
    for new in ([300, 77], [1, 1], [1, 1], [1, 1]):
        batch = seqs.extend(new)
        x = torch.randn(sum(new), 2048, device=device).bfloat16()
        y = layer(x, seqs.cache, batch)
        print(f"{new} new tokens, lengths {seqs.lengths}: out {tuple(y.shape)}, "
              f"rms {y.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
