"""Generation through one attention block of a quantized model: prompts in
chunks, then one token at a time for the whole batch.

Every step is the library's: the q/k/v linears (frozen 4-bit weights with
their adapters) in one grouped call, rotary positions, keys and values
quantized into the paged cache as they are written, attention of the new
tokens over it, and the output linear.

    python examples/attention_block.py [--width 4096] [--heads 32] [--kv-heads 8] [--kv int8] [--prompt 300]
                                       [--batch 4] [--steps 16]

Weights and inputs are random; the run prints the time of a decoding step and
checks that decoding gives what running the same tokens as one prompt gives.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bit_nf4_quantized_21_amd as qlora  # noqa: E402


class AttentionBlock:
    """q/k/v/o linears of `width`, a paged cache of `pages` pages, rotary
    positions up to `positions`."""

    def __init__(self, width, heads, kv_heads, kv="int8", pages=256, page_size=32, positions=4096, rank=16, seed=0):
        self.heads, self.kv_heads, self.dim, self.rank, self.alpha = heads, kv_heads, width // heads, rank, 16.0
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.linears = {}
        for name, n in (("q", width), ("k", kv_heads * self.dim), ("v", kv_heads * self.dim), ("o", width)):
            w = torch.randn(n, width, generator=g, device="cuda") * 0.02
            codes, q8, s2 = qlora.quantize_dq(w)
            a = (torch.rand(width, rank, generator=g, device="cuda") * 2 - 1) * width ** -0.5
            b = torch.randn(rank, n, generator=g, device="cuda") * 0.01
            self.linears[name] = dict(codes=codes, q8=q8, s2=s2, A=a.bfloat16(), B=b.bfloat16())
        self.cache = qlora.KVCache.empty(pages, kv_heads, page_size, self.dim, kv_type=kv)
        self.table = qlora.rope_table(positions, self.dim)

    def __call__(self, x, positions, slots, pages, starts, lengths, max_new, max_len):
        """x: bf16 [tokens, width] of all sequences in a row; the rest as
        attend_paged and kv_write take it."""
        tokens = x.shape[0]
        (q, _), (k, _), (v, _) = qlora.linear_fwd_grouped([dict(self.linears[n], X=x) for n in "qkv"], self.alpha,
                                                          tokens, self.rank)
        q = q.view(tokens, self.heads, self.dim)
        k, v = (t.view(tokens, self.kv_heads, self.dim) for t in (k, v))
        qlora.kv_write(self.cache, k, v, slots, table=self.table, positions=positions)
        qlora.rope(q, None, self.table, positions, q_out=q)
        out, _ = qlora.attend_paged(q, self.cache, pages, starts, lengths, max_new, max_len)
        o = self.linears["o"]
        y, _ = qlora.linear_fwd(out.view(tokens, -1), o["codes"], o["q8"], o["s2"], o["A"], o["B"], self.alpha, x.shape[1])
        return y


class Sequences:
    """Pages and lengths of a batch: every sequence gets pages as it grows."""

    def __init__(self, batch, page_size, pages):
        self.page_size, self.free = page_size, list(range(pages))
        self.held = [[] for _ in range(batch)]
        self.length = [0] * batch

    def extend(self, new):
        """Room for new[b] tokens of each sequence; what a call needs, on the GPU."""
        positions, slots, starts = [], [], [0]
        for b, n in enumerate(new):
            for p in range(self.length[b], self.length[b] + n):
                if p // self.page_size == len(self.held[b]):
                    self.held[b].append(self.free.pop())
                positions.append(p)
                slots.append(self.held[b][p // self.page_size] * self.page_size + p % self.page_size)
            self.length[b] += n
            starts.append(starts[-1] + n)
        width = max(len(h) for h in self.held)
        table = [h + [0] * (width - len(h)) for h in self.held]
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(positions=torch.tensor(positions, **i32), slots=torch.tensor(slots, device="cuda"),
                    pages=torch.tensor(table, **i32), starts=torch.tensor(starts, **i32),
                    lengths=torch.tensor(self.length, **i32), max_new=max(new), max_len=max(self.length))


def run(width=4096, heads=32, kv_heads=8, kv="int8", prompt=300, batch=4, steps=16, chunk=128, page_size=32, seed=0):
    """(outputs of the decoded tokens, the same tokens' outputs when each
    sequence is given whole, seconds per decoding step), outputs [batch, steps,
    width] fp32."""
    prompts = [max(1, prompt - 37 * b) for b in range(batch)]
    pages = sum((p + steps) // page_size + 1 for p in prompts)
    block = AttentionBlock(width, heads, kv_heads, kv, pages, page_size, positions=prompt + steps, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = [torch.randn(p + steps, width, generator=g, device="cuda").bfloat16() for p in prompts]
    seqs = Sequences(batch, page_size, pages)
    while any(length < p for length, p in zip(seqs.length, prompts)):
        at = list(seqs.length)
        new = [min(chunk, p - length) for length, p in zip(at, prompts)]
        block(torch.cat([t[a:a + n] for t, a, n in zip(x, at, new)]), **seqs.extend(new))
    decoded = []
    torch.cuda.synchronize()
    began = time.perf_counter()
    for i in range(steps):
        decoded.append(block(torch.stack([t[p + i] for t, p in zip(x, prompts)]), **seqs.extend([1] * batch)))
    torch.cuda.synchronize()
    seconds = (time.perf_counter() - began) / steps
    whole = Sequences(batch, page_size, pages)
    new = [p + steps for p in prompts]
    y = block(torch.cat(x), **whole.extend(new))
    ends = torch.tensor(new).cumsum(0).tolist()
    return (torch.stack(decoded, 1).float(), torch.stack([y[e - steps:e] for e in ends]).float(), seconds)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("width", 4096), ("heads", 32), ("kv-heads", 8), ("prompt", 300), ("batch", 4), ("steps", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--kv", default="int8", choices=sorted(qlora.KV_TYPES))
    a = ap.parse_args()
    decoded, whole, seconds = run(a.width, a.heads, a.kv_heads, a.kv, a.prompt, a.batch, a.steps)
    off = ((decoded - whole).norm() / whole.norm()).item()
    qlora.device_status()
    print(f"{a.batch} sequences of up to {a.prompt + a.steps} tokens, {a.kv} cache: {seconds * 1e6:.0f} us per decoding "
          f"step; decoded against whole: relative difference {off:.1e}")


if __name__ == "__main__":
    main()
