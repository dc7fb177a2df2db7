"""The cross entropy of logits that are far from zero, large or infinite, against 64 bits."""
from __future__ import annotations

import pytest
import torch

import dense_reference as ref
import tensor_core_loop_gb300 as tcl
from test_gpu_dense import far_logits, tokens_of

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


def losses(x, w, y):
    """By the call without gradients and by the one with them."""
    return tcl.cross_entropy(x, w, y), tcl.cross_entropy_grad(x, w, y, torch.ones(x.shape[0], device=DEV))


@pytest.mark.parametrize("tokens", [7, 100, 200, 2100])
@pytest.mark.parametrize("level", [100.0, 300.0, -300.0])
def test_infinite_logit_beside_far_ones(tokens, level):
    """One token with one logit of infinity, the other words' logits so far from zero that their exponentials are
    taken relative to another power of two than the infinite one."""
    x, w, y, _ = tokens_of(41, tokens, 64, 500, drop=0.0)
    x[:, :2], w[:, :2] = 0.0, 0.0
    x[:, 0] = -1.0
    x[3, 0], w[7, 0] = 1.0, INF
    x[3, 1], w[8:, 1] = level, 1.0
    y = torch.where(y == 7, 8, y)
    others = torch.arange(tokens, device=DEV) != 3
    for loss, lse, *grads in losses(x, w, y):
        assert float(lse[3]) == INF and float(loss[3]) == INF
        assert lse[others].isfinite().all() and loss[others].isfinite().all()
        if grads:
            assert grads[0][3].isnan().all() and grads[1].isnan().all()
            assert grads[0][others][:, 1:].isfinite().all()


@pytest.mark.parametrize("tokens", [7, 100, 200, 2100])
def test_logits_beyond_2_30_are_infinite(tokens):
    """Finite ones as well: two fp32 numbers there differ by more than any exponential tells, and their multiples of
    log2(e) by whole powers of two. Tokens of one large logit each, positive and negative ones in turn."""
    x = torch.zeros(tokens, 64, dtype=BF16, device=DEV)
    w = torch.zeros(300, 64, dtype=BF16, device=DEV)
    w[7, 0] = 2.0 ** 20
    w[:, 1] = (torch.arange(300, device=DEV) % 16).to(BF16)
    x[:, 1] = 1.0
    large = 2.0 ** torch.linspace(10.01, 100, tokens, device=DEV)
    x[:, 0] = (large * torch.where(torch.arange(tokens, device=DEV) % 2 == 0, 1.0, -1.0)).to(BF16)
    y = torch.full((tokens,), 20, device=DEV)
    up = x[:, 0] > 0
    keep = torch.arange(300, device=DEV) != 7
    want = torch.logsumexp(w[keep, 1].double(), 0)
    for loss, lse, *grads in losses(x, w, y):
        assert (lse[up] == INF).all() and (loss[up] == INF).all()
        assert ((lse[~up] - want).abs() <= 2.0 ** -20 * want).all() and loss[~up].isfinite().all()
        if grads:
            assert grads[0][up].isnan().all()


@pytest.mark.parametrize("tokens", [16, 300, 2100])
@pytest.mark.parametrize("level", [-1e5, -1e7, -1e8, -5e8, 1e7, 5e8])
def test_targets_far_above_the_rest_at_any_level(tokens, level):
    """The target's logit, summed a second time, is off from the tensor core's by more than one: what that takes from
    the sum of exponentials may not be more than there is."""
    g = torch.Generator().manual_seed(42)
    x = torch.rand(tokens, 4096, generator=g) + 0.5
    w = (torch.rand(300, 1, generator=g) * 0.5 + 1.0) * (1 + 0.01 * torch.rand(300, 4096, generator=g))
    x = x.to(BF16).to(DEV)
    w = (w * (level / 4096)).to(BF16).to(DEV)
    l = x.double() @ w.double().t()
    y = l.argmax(1)
    want = ref.cross_entropy(x, w, y)
    for loss, lse, *grads in losses(x, w, y):
        ref.within(lse, want[1], "lse")
        ref.within(loss, want[0], "loss")
        assert (loss >= -2.0 ** -22 * lse.abs()).all()
        assert all(t.isfinite().all() for t in grads)


@pytest.mark.parametrize("level,spread", [(40.0, 1.0), (64.0, 8.0), (90.0, 1.0), (300.0, 20.0), (20000.0, 1.0)])
def test_logits_far_from_zero_of_many_tokens(level, spread):
    """More than 2048 tokens: eight rows to a block of the pass that brings a row's exponentials to one power of two."""
    x, w, y, grad = far_logits(43, 2100, 1100, level, spread)
    want = ref.cross_entropy(x, w, y, grad)
    for got in (tcl.cross_entropy(x, w, y), tcl.cross_entropy_grad(x, w, y, grad)):
        for g, r, what in zip(got, want, ("loss", "lse", "dx", "dw")):
            ref.within(g, r, what)
