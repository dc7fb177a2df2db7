"""A mixture-of-experts feed-forward layer in e4m3 on the library's calls.

Each token's `top` experts compute  W_out[e] · (silu(g) * u),  (g, u) = W_in[e] · x , and the
token's output is their sum with the router's weights. All products of both directions run on
the 8-bit tensor cores, with one fp32 scale for each 128 values of the activations and for each
128 x 128 block of the weights; activations between the calls are bf16, weight gradients and the
master weights fp32.

    python examples/expert_layer.py          # gradients against fp32, a short training run, one serving step
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_core_loop_gb300 as tcl  # noqa: E402


class ExpertLayer:
    def __init__(self, experts: int, hidden: int, inner: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.experts = experts
        self.w_in = torch.randn(experts, 2 * inner, hidden, device=device, generator=g) * hidden ** -0.5
        self.w_out = torch.randn(experts, hidden, inner, device=device, generator=g) * inner ** -0.5
        self.quantize()

    def quantize(self):
        """The weights as the products read them; once after each update."""
        self.q_in = tcl.quantize_fp8(self.w_in, along="blocks")
        self.q_out = tcl.quantize_fp8(self.w_out, along="blocks")

    def forward(self, x, ids, weights, train: bool = False):
        """x: tokens x hidden (bf16); ids, weights: tokens x top. Serving keeps the experts' rows close
        together; training pads them so that no group of 128 rows spans two experts."""
        order = tcl.sort_by_expert(ids, self.experts, align=128 if train else 1)
        h = tcl.gemm_fp8_experts(*tcl.quantize_fp8(x, order=order), *self.q_in, order.offsets)
        gate, up = h.chunk(2, -1)
        a = F.silu(gate) * up
        y = tcl.gemm_fp8_experts(*tcl.quantize_fp8(a), *self.q_out, order.offsets)
        out = tcl.combine(y, weights, order)
        return (out, (x, weights, order, h, a, y)) if train else out

    def backward(self, grad, saved):
        """(gradients of x, of the router's weights, of w_in, of w_out) from the output's (bf16)."""
        x, weights, order, h, a, y = saved
        off = order.offsets
        dy, d_weights = tcl.combine_grad(grad, y, weights, order)
        da = tcl.gemm_fp8_experts(*tcl.quantize_fp8(dy), *tcl.quantize_fp8(self.w_out, along="blocks_t"), off)
        d_out = tcl.gemm_fp8_experts_wgrad(*tcl.quantize_fp8(dy, along="columns"),
                                           *tcl.quantize_fp8(a, along="columns"), off, out_dtype=torch.float32)
        gate, up = (t.float() for t in h.chunk(2, -1))
        s = torch.sigmoid(gate)
        dh = torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], -1).to(torch.bfloat16)
        dx = tcl.gemm_fp8_experts(*tcl.quantize_fp8(dh), *tcl.quantize_fp8(self.w_in, along="blocks_t"), off)
        d_in = tcl.gemm_fp8_experts_wgrad(*tcl.quantize_fp8(dh, along="columns"),
                                          *tcl.quantize_fp8(x, along="columns", order=order), off,
                                          out_dtype=torch.float32)
        return tcl.combine(dx, None, order), d_weights, d_in, d_out


def plain(layer, x, ids, weights):
    """The layer in fp32, expert by expert (for autograd)."""
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (x[t] @ layer.w_in[e].t()).chunk(2, -1)
        out = out.index_add(0, t, weights[t, j, None] * ((F.silu(gate) * up) @ layer.w_out[e].t()))
    return out


def router(tokens, experts, top, device, seed):
    g = torch.Generator(device=device).manual_seed(seed)
    best, ids = torch.randn(tokens, experts, device=device, generator=g).topk(top, -1)
    return ids, torch.softmax(best, -1)


def distances(tokens=300, experts=6, top=2, hidden=384, inner=256, device="cuda"):
    """Relative 2-norm distances of output and gradients from fp32 autograd."""
    layer = ExpertLayer(experts, hidden, inner, device)
    ids, weights = router(tokens, experts, top, device, 1)
    ids[::17] = -1                                        # padding tokens go nowhere
    g = torch.Generator(device=device).manual_seed(2)
    x = torch.randn(tokens, hidden, device=device, generator=g).to(torch.bfloat16)
    grad = torch.randn(tokens, hidden, device=device, generator=g).to(torch.bfloat16)
    out, saved = layer.forward(x, ids, weights, train=True)
    got = (out, *layer.backward(grad, saved))
    leaves = [t.detach().float().requires_grad_() for t in (x, weights, layer.w_in, layer.w_out)]
    ref = ExpertLayer.__new__(ExpertLayer)
    ref.experts, ref.w_in, ref.w_out = experts, leaves[2], leaves[3]
    want = plain(ref, leaves[0], ids, leaves[1])
    want.backward(grad.float())
    exact = [want.detach()] + [t.grad for t in leaves]
    names = ("output", "x", "router weights", "w_in", "w_out")
    return {n: float((u.float() - v).norm() / v.norm()) for n, u, v in zip(names, got, exact)}


def train(steps=60, tokens=2048, experts=8, top=2, hidden=512, inner=512, lr=0.03, device="cuda"):
    """Fits the layer to another one's outputs; the losses."""
    teacher = ExpertLayer(experts, hidden, inner, device, seed=7)
    layer = ExpertLayer(experts, hidden, inner, device, seed=0)
    layer.w_in.copy_(teacher.w_in + 0.5 * layer.w_in)
    layer.w_out.copy_(teacher.w_out + 0.5 * layer.w_out)
    layer.quantize()
    losses = []
    for step in range(steps):
        ids, weights = router(tokens, experts, top, device, 100 + step)
        x = torch.randn(tokens, hidden, device=device).to(torch.bfloat16)
        target = teacher.forward(x, ids, weights)
        out, saved = layer.forward(x, ids, weights, train=True)
        diff = out.float() - target.float()
        losses.append(diff.square().mean())
        _, _, d_in, d_out = layer.backward((diff * (2 * experts / (tokens * top))).to(torch.bfloat16), saved)
        layer.w_in -= lr * d_in
        layer.w_out -= lr * d_out
        layer.quantize()
    return [float(v) for v in losses]


def main():
    torch.manual_seed(0)
    for name, d in distances().items():
        print(f"{name:15s} relative distance from fp32 {d:.4f}")
    losses = train()
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    layer = ExpertLayer(64, 4096, 2048)
    ids, weights = router(16, 64, 8, "cuda", 3)
    x = torch.randn(16, 4096, device="cuda").to(torch.bfloat16)
    layer.forward(x, ids, weights)                        # kernels are loaded outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, ids, weights)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"serving: 16 tokens, 64 experts of 4096 x 2048, {begin.elapsed_time(end) / 20 * 1e3:.1f} us a step (CUDA graph)")
    print("device status", tcl.last_device_error())


if __name__ == "__main__":
    main()
