"""The gated feed-forward block, the cross entropy over a vocabulary and their gradients on the GPU,
value by value against 64 bits, at the sizes, layouts and values where they can go wrong."""
from __future__ import annotations

import pytest
import torch

import dense_reference as ref
import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


def laid_out(v, pitch=None, offset=0):
    """v (bf16) with rows `pitch` apart, `offset` elements behind an aligned address; NaN around it."""
    rows, cols = v.shape
    pitch = pitch or cols
    room = torch.full((offset + max(rows - 1, 0) * pitch + cols + 64,), float("nan"), dtype=BF16, device=DEV)
    view = room.as_strided((rows, cols), (pitch, 1), offset)
    view.copy_(v)
    return view


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(BF16).to(DEV)


def block(seed, tokens, hidden, inner):
    g = torch.Generator().manual_seed(seed)
    return (normal(g, tokens, hidden), normal(g, inner, hidden, scale=hidden ** -0.5),
            normal(g, inner, hidden, scale=hidden ** -0.5), normal(g, hidden, inner, scale=inner ** -0.5),
            normal(g, tokens, hidden))


# ------------------------------------------------------------------------------ the feed-forward block

SIZES = [(1, 1, 1), (1, 64, 128), (1, 8, 8), (2, 72, 56), (16, 256, 384), (17, 130, 70), (32, 512, 1000), (33, 1030, 515),
         (64, 320, 4100), (65, 256, 384), (128, 64, 64), (256, 128, 256), (257, 1030, 777), (300, 776, 2056), (513, 65, 129),
         (700, 192, 1000)]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,hidden,inner", SIZES)
def test_ffn(tokens, hidden, inner, act):
    x, wg, wu, wd, grad = block(tokens + hidden, tokens, hidden, inner)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, activation=act, keep=True)
    want = ref.gated_ffn(x, wg, wu, wd, act)
    for got, w, what in zip((out, *kept), want, ("out", "gate", "up", "hidden")):
        assert got.dtype == BF16
        ref.within(got, w, what)
    assert torch.equal(tcl.gated_ffn(x, wg, wu, wd, activation=act), out)
    got = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, activation=act)
    for g, w, what in zip(got, ref.gated_ffn_grad(grad, x, wg, wu, wd, act), ("dx", "dw_gate", "dw_up", "dw_down")):
        assert g.dtype == BF16
        ref.within(g, w, what)


# ------------------------------------------------------------------------------ the cross entropy

def tokens_of(seed, tokens, hidden, vocab, spread=1.5, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(vocab, hidden, generator=g) * spread * hidden ** -0.5
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x = torch.randn(tokens, hidden, generator=g)
    x += 10 * torch.rand(tokens, 1, generator=g) * w[y] / (w[y] ** 2).sum(1, keepdim=True).clamp_min(1e-3)
    y[torch.rand(tokens, generator=g) < drop] = -100
    grad = torch.rand(tokens, generator=g) / tokens
    return x.to(BF16).to(DEV), w.to(BF16).to(DEV), y.to(DEV), grad.to(DEV)


ENTROPY_SIZES = [(1, 1, 1), (1, 64, 1), (1, 64, 500), (3, 8, 31), (16, 256, 5000), (17, 130, 1001), (33, 72, 129), (64, 1030, 700),
                 (65, 128, 64), (100, 64, 128), (256, 320, 4096), (257, 130, 3001), (300, 65, 20011), (1000, 512, 257)]


@pytest.mark.parametrize("ids", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,hidden,vocab", ENTROPY_SIZES)
def test_entropy(tokens, hidden, vocab, ids):
    x, w, y, grad = tokens_of(tokens + vocab, tokens, hidden, vocab)
    loss, lse = tcl.cross_entropy(x, w, y.to(ids))
    want = ref.cross_entropy(x, w, y)
    ref.within(loss, want[0], "loss")
    ref.within(lse, want[1], "lse")
    got = tcl.cross_entropy_grad(x, w, y.to(ids), grad)
    want = ref.cross_entropy(x, w, y, grad)
    kept = y >= 0
    ref.within(got[0], want[0], "loss")
    ref.within(got[1][kept], ref.V(want[1].v[kept], want[1].e[kept]), "lse")
    ref.within(got[2], want[2], "dx")
    ref.within(got[3], want[3], "dw")
