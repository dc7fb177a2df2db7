"""The example of a dense block on the GPU: it runs, captured too, and its gradients are those of 64 bits."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import dense_reference as ref
import tensor_core_loop_gb300 as tcl

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from dense_block import DenseBlock  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


def tokens(seed, n, hidden, vocab):
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, vocab, (n,), generator=g)
    y[::5] = -100
    return torch.randn(n, hidden, generator=g).to(torch.bfloat16).to(DEV), y.to(DEV)


@pytest.mark.parametrize("n,hidden,inner,vocab,act", [(33, 72, 130, 501, "gelu"), (300, 256, 704, 1000, "silu")])
def test_gradients(n, hidden, inner, vocab, act):
    """Each call's results against 64 bits of what it was given."""
    block = DenseBlock(hidden, inner, vocab, activation=act)
    x, y = tokens(1, n, hidden, vocab)
    grad = torch.rand(n, generator=torch.Generator().manual_seed(2)).to(DEV) / n
    loss, dx, grads = block.gradients(x, y, grad)
    gate, up, down, table = block.weights
    hidden_states = x + tcl.gated_ffn(x, gate, up, down, activation=act)
    want = ref.cross_entropy(hidden_states, table, y, grad)
    ref.within(loss, want[0], "loss")
    ref.within(grads[3], want[3], "table")
    dy = tcl.cross_entropy_grad(hidden_states, table, y, grad)[2]
    ref.within(dy, want[2], "dy")
    for got, w, what in zip(grads, ref.gated_ffn_grad(dy, x, gate, up, down, act)[1:], ("gate", "up", "down")):
        ref.within(got, w, what)
    through = ref.gated_ffn_grad(dy, x, gate, up, down, act)[0]
    ref.within(dx, ref.rounded(ref.plus(ref.exactly(dy), through)), "dx")


def test_it_runs_and_is_captured():
    block, twin = DenseBlock(128, 200, 333), DenseBlock(128, 200, 333)
    x, y = tokens(3, 70, 128, 333)
    step, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    block.train_step(x, y)   # (both start one step on: what the allocator and the library set up once is in place)
    twin.train_step(x, y)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(step, stream=stream):
        held = twin.train_step(x, y)
    for _ in range(3):
        loss, norm = block.train_step(x, y)
        step.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, held[0]) and torch.equal(norm, held[1])
        assert all(torch.equal(a, b) for a, b in zip(block.weights, twin.weights))
    assert block.evaluate(x[1:2], y[1:2]).isfinite().all() and block.serve(x[:1]).shape == (1, 128)
