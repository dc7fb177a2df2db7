"""A language model's last block on the dense calls: residual gated feed-forward, logits over a vocabulary,
cross entropy, gradients, clipping, and a plain gradient step; evaluation and a step of serving.

    python examples/dense_block.py
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import tensor_core_loop_gb300 as tcl  # noqa: E402


class DenseBlock:
    """y = x + ffn(x), logits y · tableᵀ. Weights in bf16 with fp32 masters."""

    def __init__(self, hidden: int, inner: int, vocab: int, seed: int = 0, device="cuda:0", activation: str = "silu"):
        g = torch.Generator().manual_seed(seed)
        shapes = ((inner, hidden), (inner, hidden), (hidden, inner), (vocab, hidden))
        self.masters = [(torch.randn(*s, generator=g) * s[1] ** -0.5).to(device) for s in shapes]
        self.weights = [m.to(torch.bfloat16) for m in self.masters]
        self.activation = activation

    def gradients(self, x, targets, grad):
        """(each token's loss, gradient of x, gradients of the weights) of Σ grad · loss."""
        gate, up, down, table = self.weights
        out, kept = tcl.gated_ffn(x, gate, up, down, activation=self.activation, keep=True)
        y = x + out
        loss, _, dy, dtable = tcl.cross_entropy_grad(y, table, targets, grad)
        dx, *dw = tcl.gated_ffn_grad(dy, x, gate, up, down, kept, activation=self.activation)
        return loss, dy + dx, [*dw, dtable]

    def train_step(self, x, targets, rate: float = 0.5, max_norm: float = 1.0):
        """One step on the tokens whose targets are in the vocabulary; (mean loss, gradient norm), on the GPU."""
        learnt = ((targets >= 0) & (targets < self.masters[3].shape[0])).float()
        grad = learnt / learnt.sum().clamp_min(1.0)
        loss, _, grads = self.gradients(x, targets, grad)
        norm = tcl.clip_grads(grads, max_norm)
        for master, weight, d in zip(self.masters, self.weights, grads):
            master.sub_(d, alpha=rate)
            weight.copy_(master)
        return (loss * grad).sum(), norm

    def evaluate(self, x, targets):
        """Each token's loss."""
        return tcl.cross_entropy(self.serve(x), self.weights[3], targets)[0]

    def serve(self, x):
        """The hidden states behind the block."""
        gate, up, down, _ = self.weights
        return x + tcl.gated_ffn(x, gate, up, down, activation=self.activation)


def main() -> None:
    block = DenseBlock(512, 1408, 4000)
    g = torch.Generator(device="cuda:0").manual_seed(1)
    x = torch.randn(1000, 512, device="cuda:0", generator=g).to(torch.bfloat16)
    targets = torch.randint(0, 4000, (1000,), device="cuda:0", generator=g)
    targets[::10] = -100   # (a prompt's tokens: nothing is learnt from them)
    for step in range(10):
        loss, norm = block.train_step(x, targets)
        print(f"step {step}: loss {float(loss):.3f}, gradient norm {float(norm):.3f}")
    print(f"loss of the first token: {float(block.evaluate(x[1:2], targets[1:2])[0]):.3f}")


if __name__ == "__main__":
    main()
