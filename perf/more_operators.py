"""Measured cases of a language model's dense training and serving path on bf16 matrices.

Three kinds of call:

ffn        the gated feed-forward block, out = (act(x·Wg^T) * (x·Wu^T))·Wd^T; in training also the
           gradients of x and of the three matrices
entropy    softmax cross entropy of the logits x·W^T over a vocabulary, which are never kept: each
           token's loss and log-sum-exp; in training also the gradients of x and of W
clip       the norm over all gradients of a model, and the gradients scaled down to a bound on it

`run` computes them in plain fp32 operations, or, where `own` is set, by the package's entry points.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
LONGEST_EXACT = 1.2e13     # operations in 64 bits that fit into some ten seconds


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one sequence, one token: the weights' way through the memory
        dict(name="ffn 1 token", op="ffn", tokens=1, hidden=4096, inner=14336, act="silu", train=False),
        # one step of serving 16 sequences
        dict(name="ffn 16 tokens", op="ffn", tokens=16, hidden=4096, inner=14336, act="silu", train=False),
        # a prompt, ragged everywhere: rows off the 16-byte grid, tiles cut at every edge
        dict(name="ffn 1000 tokens odd", op="ffn", tokens=1000, hidden=1030, inner=2777, act="gelu", train=False),
        # a batch of prompts
        dict(name="ffn 8192 tokens", op="ffn", tokens=8192, hidden=4096, inner=14336, act="silu", train=False),
        # a small training step, ragged
        dict(name="ffn 777 tokens train", op="ffn", tokens=777, hidden=776, inner=2056, act="gelu", train=True),
        # a training batch, forward and backward
        dict(name="ffn 4096 tokens train", op="ffn", tokens=4096, hidden=4096, inner=14336, act="silu", train=True),
        # the likelihood of a short continuation
        dict(name="entropy 16 tokens", op="entropy", tokens=16, hidden=4096, vocab=131072, train=False),
        # evaluation of a text, an odd vocabulary
        dict(name="entropy 2047 tokens", op="entropy", tokens=2047, hidden=2048, vocab=50001, train=False),
        # a small training step, ragged everywhere
        dict(name="entropy 1023 tokens train", op="entropy", tokens=1023, hidden=1030, vocab=32001, train=True),
        # a training batch over a large vocabulary
        dict(name="entropy 8192 tokens train", op="entropy", tokens=8192, hidden=4096, vocab=131072, train=True),
        # a small model's fp32 gradients: many short tensors
        dict(name="clip 62 fp32 tensors", op="clip", count=62, total=1_000_003, dtype="f32", bound=1.0, norm=7.0),
        # a shard of a large model's bf16 gradients
        dict(name="clip 18 bf16 tensors", op="clip", count=18, total=1_000_000_000, dtype="bf16", bound=1.0, norm=3.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A matrix width: mostly whole groups of 64, now and then an odd one."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(64, (v + 32) // 64 * 64)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn", "entropy", "entropy", "clip"])
    train = rng.random() < 0.5
    if op == "ffn":
        return dict(op=op, tokens=_log(rng, 1, 4096 if train else 8192), hidden=_width(rng, 128, 4096),
                    inner=_width(rng, 128, 14336), act=rng.choice(["silu", "silu", "gelu"]), train=train)
    if op == "entropy":
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=_width(rng, 128, 4096), vocab=_width(rng, 500, 131072),
                    train=train)
    return dict(op=op, count=rng.randint(1, 62), total=_log(rng, 1000, 1_000_000_000), dtype=rng.choice(["bf16", "f32"]),
                bound=1.0, norm=rng.choice([0.25, 3.0, 40.0]))


def _sizes(case):
    """Lengths of a model's gradients: vectors between matrices that share the rest, `total` in all."""
    count, total = case["count"], case["total"]
    short = [min(4096 + 7 * i, max(1, total // (8 * count))) if i % 3 == 2 else 0 for i in range(count)]
    long = sum(n == 0 for n in short)
    rest = total - sum(short)
    sizes, at = [], 0
    for n in short:
        if not n:
            at += 1
            n = rest * at // long - rest * (at - 1) // long
        sizes.append(n)
    return sizes


def work(case):
    op = case["op"]
    if op == "clip":
        each = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * each * case["total"] + 4, "flops": 3 * case["total"]}
    t, h = case["tokens"], case["hidden"]
    if op == "ffn":
        f = case["inner"]
        if not case["train"]:
            return {"bytes": 2 * (2 * t * h + 3 * h * f), "flops": 6 * t * h * f}
        # in: x, the result's gradient, the matrices; out: the result and the four gradients
        return {"bytes": 2 * (4 * t * h + 6 * h * f), "flops": 18 * t * h * f}
    v = case["vocab"]
    if not case["train"]:
        return {"bytes": 2 * (t * h + v * h) + 16 * t, "flops": 2 * t * h * v}
    return {"bytes": 4 * (t * h + v * h) + 20 * t, "flops": 6 * t * h * v}


# ------------------------------------------------------------------------------ plain forms

def _gate(g, act):
    """(activation of g, its derivative)"""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_ffn(s, act, train):
    x, wg, wu, wd = (s[k].float() for k in ("x", "gate", "up", "down"))
    g, u = x @ wg.t(), x @ wu.t()
    a, slope = _gate(g, act)
    h = a * u
    out = (h @ wd.t()).to(BF16)
    if not train:
        return out
    grad = s["grad"].float()
    dh = grad @ wd
    dg, du = dh * u * slope, dh * a
    dx = dg @ wg + du @ wu
    return out, dx.to(BF16), (dg.t() @ x).to(BF16), (du.t() @ x).to(BF16), (grad.t() @ h).to(BF16)


def _plain_entropy(s, train):
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    kept = (targets >= 0) & (targets < w.shape[0])
    at = targets.clamp(0, w.shape[0] - 1)[:, None]
    loss = torch.where(kept, lse - logits.gather(1, at)[:, 0], 0.0)
    if not train:
        return loss, lse
    d = torch.exp(logits - lse[:, None])
    d.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    d *= torch.where(kept, s["grad"], 0.0)[:, None]
    return loss, lse, (d @ w).to(BF16), (d.t() @ x).to(BF16)


def _plain_clip(s, bound):
    squares = [(g.float() ** 2).sum(dtype=torch.float64) for g in s["grads"]]
    norm = torch.stack(squares).sum().sqrt().float()
    scale = torch.where(norm > bound, bound / norm, torch.ones_like(norm))
    return norm, [(g.float() * scale).to(g.dtype) for g in s["grads"]]


def _plain(s):
    c = s["case"]
    if c["op"] == "ffn":
        return _plain_ffn(s, c["act"], c["train"])
    if c["op"] == "entropy":
        return _plain_entropy(s, c["train"])
    return _plain_clip(s, c["bound"])


# ------------------------------------------------------------------------------ the package's calls

def _own(s):
    import tensor_core_loop_gb300 as tcl
    c = s["case"]
    if c["op"] == "ffn":
        w = s["gate"], s["up"], s["down"]
        if not c["train"]:
            return tcl.gated_ffn(s["x"], *w, activation=c["act"])
        out, kept = tcl.gated_ffn(s["x"], *w, activation=c["act"], keep=True)
        return (out,) + tuple(tcl.gated_ffn_grad(s["grad"], s["x"], *w, kept, activation=c["act"]))
    if c["op"] == "entropy":
        if not c["train"]:
            return tcl.cross_entropy(s["x"], s["w"], s["targets"])
        return tcl.cross_entropy_grad(s["x"], s["w"], s["targets"], s["grad"])
    norm = tcl.clip_grads(s["grads"], c["bound"], out=s["out"])
    return norm, s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------ inputs

def _hidden(gen, rows, cols):
    """Normalised hidden states: near normal, a few channels ten times as large."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    loud = torch.rand(cols, device="cuda", generator=gen) < 0.01
    return x * torch.where(loud, 4.0, 1.0)


def _matrix(gen, rows, cols):
    """A weight matrix whose products with hidden states are of the size of one."""
    return (torch.randn(rows, cols, device="cuda", generator=gen) * (1.0 / math.sqrt(cols))).to(BF16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "clip":
        dtype = BF16 if case["dtype"] == "bf16" else F32
        each = case["norm"] / math.sqrt(case["total"])
        s["grads"] = [(torch.randn(n, device="cuda", generator=gen) * each).to(dtype) for n in _sizes(case)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        return s
    t, h = case["tokens"], case["hidden"]
    if op == "ffn":
        s["x"] = _hidden(gen, t, h).to(BF16)
        s["gate"], s["up"] = _matrix(gen, case["inner"], h), _matrix(gen, case["inner"], h)
        s["down"] = _matrix(gen, h, case["inner"])
        if case["train"]:
            s["grad"] = (torch.randn(t, h, device="cuda", generator=gen) / t).to(BF16)
        return s
    v = case["vocab"]
    # logits spread by 1.5, and the model likes a token's target by up to a dozen more
    w = torch.randn(v, h, device="cuda", generator=gen) * (1.5 / math.sqrt(h))
    targets = torch.randint(0, v, (t,), device="cuda", generator=gen)
    liked = 12.0 * torch.rand(t, 1, device="cuda", generator=gen)
    s["x"] = (_hidden(gen, t, h) + liked * w[targets] / (w[targets] ** 2).sum(1, keepdim=True)).to(BF16)
    s["w"] = w.to(BF16)
    # prompts and padding are not learnt from: their targets are -100
    s["targets"] = torch.where(torch.rand(t, device="cuda", generator=gen) < 0.05, -100, targets)
    if case["train"]:
        learnt = (s["targets"] >= 0).float()
        s["grad"] = learnt / learnt.sum().clamp_min(1.0)
    return s


# ------------------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if work(case)["flops"] > LONGEST_EXACT:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        scale = min(1.0, case["bound"] / norm) if norm else 1.0
        return torch.tensor(norm, dtype=torch.float64), [g.double() * scale for g in s["grads"]]
    with torch.enable_grad():
        if op == "ffn":
            x, wg, wu, wd = (s[k].double().requires_grad_(case["train"]) for k in ("x", "gate", "up", "down"))
            act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
            out = torch.nn.functional.linear(act(torch.nn.functional.linear(x, wg)) * torch.nn.functional.linear(x, wu), wd)
            if not case["train"]:
                return out
            return (out.detach(),) + torch.autograd.grad(out, (x, wg, wu, wd), s["grad"].double())
        x, w = (s[k].double().requires_grad_(case["train"]) for k in ("x", "w"))
        logits = torch.nn.functional.linear(x, w)
        lse = torch.logsumexp(logits, 1)
        loss = torch.nn.functional.cross_entropy(logits, s["targets"], ignore_index=-100, reduction="none")
        if not case["train"]:
            return loss, lse
        dx, dw = torch.autograd.grad(loss, (x, w), s["grad"].double())
        return loss.detach(), lse.detach(), dx, dw
