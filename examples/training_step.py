"""A training step of a quantized model's last block: the gated feed-forward
block with its residual, the loss over the vocabulary, the way back, clipping
and the optimizer's step.

Every step is the library's: gate and up with their activation in one call, the
down linear, the head's loss with its gradient, the backward of both, the global
norm over all adapters' gradients with the clipped values written to one flat
buffer, and AdamW on it.  The 4-bit weights and the head are frozen; the adapters
learn.

    python examples/training_step.py [--width 4096] [--features 11008] [--vocabulary 32000] [--tokens 2048]
                                     [--rank 64] [--steps 10]

Weights and inputs are random; the run prints the loss and the time of a step.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bit_nf4_quantized_21_amd as qlora  # noqa: E402


class LastBlock:
    """y = x + down(act(gate(x)) * up(x)) and the head on y, with adapters of
    `rank` whose values are views of one flat bf16 buffer."""

    NAMES = [(side, m) for side in ("gate", "up", "down") for m in "AB"]

    def __init__(self, width, features, vocabulary, rank=16, alpha=16.0, act="silu", seed=0):
        self.width, self.features, self.rank, self.alpha, self.act = width, features, rank, alpha, act
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {}
        self.linears = {}
        for name, n, k in (("gate", features, width), ("up", features, width), ("down", width, features)):
            codes, q8, s2 = qlora.quantize_dq(torch.randn(n, k, generator=g, device="cuda") * 0.02)
            self.linears[name] = dict(codes=codes, q8=q8, s2=s2)
            shapes[name, "A"], shapes[name, "B"] = (k, rank), (rank, n)
        sizes = [shapes[n][0] * shapes[n][1] for n in self.NAMES]
        self.param = torch.empty(sum(sizes), dtype=torch.bfloat16, device="cuda")
        self.grad = torch.zeros_like(self.param)     # what the optimizer reads: clipped
        self.grads = {}                              # what the backward writes
        outs, at = [], 0
        for name, size in zip(self.NAMES, sizes):
            view = self.param[at:at + size].view(shapes[name])
            scale = shapes[name][0] ** -0.5 if name[1] == "A" else 0.01
            view.copy_(torch.randn(shapes[name], generator=g, device="cuda") * scale)
            self.linears[name[0]][name[1]] = view
            self.grads[name] = torch.empty(shapes[name], dtype=torch.bfloat16, device="cuda")
            outs.append(self.grad[at:at + size].view(shapes[name]))
            at += size
        self.set = qlora.GradSet([self.grads[n] for n in self.NAMES], outs)
        self.head = (torch.randn(vocabulary, width, generator=g, device="cuda") * width ** -0.5).bfloat16()
        self.master = self.param.float()
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.step_count = 0

    def forward_backward(self, x, targets):
        """Loss (of the mean over learned tokens) and every adapter's gradient; the
        input's gradient is returned too."""
        gate, up, down = (self.linears[n] for n in ("gate", "up", "down"))
        h, saved, xa = qlora.gated_fwd(x, gate, up, self.alpha, act=self.act, save=True)
        y, ha = qlora.linear_fwd(h, down["codes"], down["q8"], down["s2"], down["A"], down["B"], self.alpha, self.width)
        y = y + x
        _, _, mean, dy = qlora.head_loss(y, self.head, targets)
        dh, _, _ = qlora.linear_bwd(dy, h, ha, down["codes"], down["q8"], down["s2"], down["A"], down["B"], self.alpha,
                                    dA=self.grads["down", "A"], dB=self.grads["down", "B"])
        dx, *_ = qlora.gated_bwd(dh, x, saved, xa, gate, up, self.alpha, dA_gate=self.grads["gate", "A"],
                                 dB_gate=self.grads["gate", "B"], dA_up=self.grads["up", "A"], dB_up=self.grads["up", "B"])
        return mean, dx + dy

    def step(self, x, targets, lr=1e-3, max_norm=1.0):
        """One step; returns (mean loss, gradient norm before clipping)."""
        mean, _ = self.forward_backward(x, targets)
        norm = qlora.clip_grads(self.set, max_norm)
        self.step_count += 1
        qlora.adamw_step(self.param, self.master, self.m, self.v, self.grad, self.step_count, lr)
        return mean, norm


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("width", 4096), ("features", 11008), ("vocabulary", 32000), ("tokens", 2048), ("rank", 64),
                          ("steps", 10)):
        p.add_argument(f"--{name}", type=int, default=default)
    a = p.parse_args()
    block = LastBlock(a.width, a.features, a.vocabulary, rank=a.rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    targets = torch.randint(0, a.vocabulary, (a.tokens,), generator=g, device="cuda")
    targets[: a.tokens // 4] = -100      # a prompt: not learned
    block.step(x, targets)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        mean, norm = block.step(x, targets)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3 / max(1, a.steps)
    qlora.device_status()
    print(f"loss {float(mean):.4f}, gradient norm {float(norm):.4f}, {ms:.2f} ms a step of {a.tokens} tokens")


if __name__ == "__main__":
    main()
