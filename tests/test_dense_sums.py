"""The target's logit as an fp32 sum of its own, and the sum of exponentials brought in line with it: what the loss
owes to either.

The tensor core truncates its fp32 sums. Here every token has the same target, the only word whose row of W is not
zero: all other logits are zeros, exactly, so that the target's alone can be off. With 1000 other words, a logit l of 5.9
to 7.5 and p the target's share of the sum S = 1000 + e^l, an error d of the logit moves a loss by

    -(1 - p)·d   where both the logit and S have it (no second sum),
    p·d          where S alone has it (a second sum, S left as it is),

and without it these remain (p at most 0.65, l·log2(e) below 11, S between 1365 and 2810, lse below 8):

    the second sum        an addition errs by half a step, 2^-24 of its result at most, with either sign: the
                          root of the sum of those squares, (1 - p) of which shows
    e^l                   2^-22 of it by the special function unit, and its argument's rounding, 2^-24·11·ln 2: p·2^-20.9
    S                     an addition of exponentials to one that holds e^l, 2^-24 of S each and with either sign: at
                          most 35 of a chunk (two sums of 16 to a block of 32, four blocks) and 16 chunks: p·sqrt(51)·2^-24
    the logarithm         a step of a value below 8: 2^-21; the loss itself, below 2: 2^-24

Where all logits are far from zero, all are off by about the same, and the loss must not see it.
"""
from __future__ import annotations

import math

import pytest
import torch

import tensor_core_loop_gb300 as tcl

BF16 = torch.bfloat16
HIDDEN, WORDS, TARGET = 16384, 1001, 300


def inputs(tokens):
    g = torch.Generator().manual_seed(51)
    w = torch.randn(HIDDEN, generator=g) / 64
    w = w.to(BF16).float()
    level = 6.0 + 1.4 * torch.rand(tokens, 1, generator=g)
    noise = torch.randn(tokens, HIDDEN, generator=g) / 4
    noise -= (noise @ w)[:, None] * w / (w @ w)
    return (noise + level * w / (w @ w)).to(BF16), w.to(BF16)


def exact(x, w):
    """(logit, loss, its target's share) in 64 bits."""
    l = x.double() @ w.double()
    lse = torch.log((WORDS - 1) + torch.exp(l))
    return l, lse - l, torch.exp(l - lse)


def chain(p, lanes):
    """Roots of the summed squares of the partial sums of an fp32 sum: 8 products at a time to each of `lanes` lanes in
    turn, the lanes' sums pairwise over a warp, the warps' one after another."""
    tokens = p.shape[0]
    lane = p.view(tokens, -1, lanes, 8).transpose(1, 2).reshape(tokens, lanes, -1).cumsum(2)
    squares = (lane ** 2).sum((1, 2))
    part = lane[:, :, -1].view(tokens, lanes // 32, 32)
    while part.shape[2] > 1:
        part = part[:, :, ::2] + part[:, :, 1::2]
        squares += (part ** 2).sum((1, 2))
    return (squares + (part[:, :, 0].cumsum(1) ** 2).sum(1)).sqrt()


def bound(x, w, share):
    """On the losses' error by norm."""
    p = x.double() * w.double()
    roots = torch.maximum(chain(p, 256), chain(p, 32))   # (few tokens: a block to each; many: a warp)
    e = (1 - share) * 2.0 ** -24 * roots + share * (2.0 ** -20.9 + math.sqrt(51) * 2.0 ** -24) + 2.0 ** -21 + 2.0 ** -24
    return float(e.norm())


def truncated(x, w, chains):
    """The logits of a tensor core that adds 16 products at a time to a sum of 24 bits and cuts off the rest; blocks of
    64 to `chains` sums in turn, those in fp32 in the end. w: one word or several."""
    sums = [torch.zeros(x.shape[0], *w.shape[:-1], dtype=torch.float64) for _ in range(chains)]
    for k in range(0, x.shape[1], 16):
        i = k // 64 % chains
        s = sums[i] + x[:, k:k + 16].double() @ w[..., k:k + 16].double().t()
        sums[i] = (s.view(torch.int64) & -(1 << 29)).view(torch.float64)   # (24 of 53 bits)
    return torch.stack(sums).float().sum(0).double()


@pytest.mark.parametrize("tokens,chains", [(16, 4), (300, 1)])
def test_the_bound_tells_losses_without_a_second_sum(tokens, chains):
    x, w = inputs(tokens)
    l, want, share = exact(x, w)
    most = bound(x, w, share)
    off = truncated(x, w, chains)
    second = (x.float() * w.float()).sum(1).double()
    s = (WORDS - 1) + torch.exp(off)
    with_both = torch.log(s + torch.exp(off) * torch.expm1(second - off)) - second
    assert float((with_both - want).norm()) <= most
    assert float((torch.log(s) - second - want).norm()) > most     # the sum of exponentials left as it is
    assert float((torch.log(s) - off - want).norm()) > most        # no second sum


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [16, 300, 2100])
def test_losses_are_off_by_fp32_roundings_alone(tokens):
    """Few tokens; a block to each; a warp to each."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x, w = inputs(tokens)
    _, want, share = exact(x, w)
    most = bound(x, w, share)
    table = torch.zeros(WORDS, HIDDEN, dtype=BF16)
    table[TARGET] = w
    x, table = x.cuda(), table.cuda()
    y = torch.full((tokens,), TARGET, device="cuda")
    for loss in (tcl.cross_entropy(x, table, y)[0], tcl.cross_entropy_grad(x, table, y, torch.ones(tokens, device="cuda"))[0]):
        off = float((loss.cpu().double() - want).norm())
        assert off <= most, (off, most)
    assert tcl.last_device_error() == (0, 0)


# ------------------------------------------------------------------------------ logits far from zero

FAR_HIDDEN, FAR_WORDS = 4096, 2000


def far_inputs(tokens, level):
    """Logits around `level` that x and W owe to a direction they share, spread by 1.5; targets up to 3 above."""
    g = torch.Generator().manual_seed(52)
    w = torch.randn(FAR_WORDS, FAR_HIDDEN, generator=g) * (1.5 / FAR_HIDDEN ** 0.5)
    y = torch.randint(0, FAR_WORDS, (tokens,), generator=g)
    x = torch.randn(tokens, FAR_HIDDEN, generator=g)
    x += 3 * torch.rand(tokens, 1, generator=g) * w[y] / (w[y] ** 2).sum(1, keepdim=True)
    d = torch.randn(FAR_HIDDEN, generator=g)
    return (x + level * d / d.norm() * FAR_HIDDEN ** 0.5 / d.norm()).to(BF16), (w + d / FAR_HIDDEN ** 0.5).to(BF16), y


def far_exact(x, w, y):
    """(target's logit, lse) in 64 bits."""
    l = x.double() @ w.double().t()
    return l.gather(1, y[:, None])[:, 0], torch.logsumexp(l, 1)


def far_bound(level, chains):
    """On the root mean square of the errors of lse and loss. A sum that grows evenly to `level` is cut off by half a
    step, 2^-24 of it, with each of its hidden/16 additions, in `chains` sums that are shorter by that: by 2^-24 ·
    hidden/32 · level / chains in all. That is the same for all words but for what sets them apart (the target and the
    others' mean: by root mean square less than an eighth of the level), and it must not show. To it come the roundings of lse, of the target's sum, of the loss and of the
    exponentials' arguments, a half step each of a number up to level + 8 + log(words)."""
    return 2.0 ** -24 * (FAR_HIDDEN / 32 * abs(level) / chains / 8 + 4 * (abs(level) + 16))


LEVELS = [-100.0, -60.0, -40.0, 60.0]


@pytest.mark.parametrize("chains", [1, 4])
@pytest.mark.parametrize("level", LEVELS)
def test_the_far_bound_tells_a_target_summed_apart_from_the_rest(level, chains):
    x, w, y = far_inputs(40, level)
    target, lse = far_exact(x, w, y)
    cut = truncated(x, w, chains)
    s = torch.logsumexp(cut, 1)
    off = target - cut.gather(1, y[:, None])[:, 0]
    apart = s + torch.log1p(torch.exp(target - off - s) * torch.expm1(off))    # the target's alone as it should be
    most = far_bound(level, chains) * 40 ** 0.5
    assert float((apart - lse).norm()) > most and float((s - lse).norm()) > most
    assert float((s + off - lse).norm()) <= most                               # all of them moved by as much


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [16, 300, 2100])
@pytest.mark.parametrize("level", LEVELS)
def test_losses_of_logits_far_from_zero(tokens, level):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x, w, y = far_inputs(tokens, level)
    target, lse = far_exact(x, w, y)
    x, w, y = x.cuda(), w.cuda(), y.cuda()
    # (few tokens without gradients: four sums in turn)
    for chains, got in ((4 if tokens <= 64 else 1, tcl.cross_entropy(x, w, y)),
                        (1, tcl.cross_entropy_grad(x, w, y, torch.ones(tokens, device="cuda")))):
        most = far_bound(level, chains) * tokens ** 0.5
        for what, value, want in (("loss", got[0], lse - target), ("lse", got[1], lse)):
            off = float((value.cpu().double() - want).norm())
            assert off <= most, (what, off, most)
    assert tcl.last_device_error() == (0, 0)
