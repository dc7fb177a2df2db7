"""Measured cases of the 8-bit floating point products and of the expert routing around them.

Six kinds of call, as a program that trains or serves a mixture-of-experts layer makes them:

quantize   a bf16 matrix to e4m3 with one fp32 scale for each 128 values: along the rows
           (activations), down the columns and stored transposed (operands of a weight
           gradient), or for each 128 x 128 block (weights)
gemm       C = A·B^T of two such matrices
experts    the same with a matrix B for each expert, over rows sorted by expert
wgrad      the experts' weight gradients, one product over each expert's own rows
route      tokens sorted by expert: the order, and the tokens' rows laid out in it (as bf16, or
           quantised on the way)
combine    the experts' rows back in token order with the router's weights applied; in training
           also the gradients of the rows and of the weights

`run` computes them in plain fp32 operations, or, where `own` is set, by the package's entry points.
"""
import math

import torch

own = False

GROUP = 128                     # values that share a scale
TOP = 448.0                     # largest e4m3 value
TINY = 2.0 ** -126              # smallest scale (an all-zero group)
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one step of serving 16 sequences: the hidden states before a projection
        dict(name="quantize rows 16x4096", op="quantize", along="rows", rows=16, cols=4096),
        # a training batch's activations, transposed for the weight gradient
        dict(name="quantize columns 16384x4096", op="quantize", along="columns", rows=16384, cols=4096),
        # one sequence, one token through a square projection
        dict(name="gemm 1x4096x4096", op="gemm", m=1, n=4096, k=4096, b="blocks", out="bf16"),
        # ragged everywhere, both operands scaled along their rows, fp32 result
        dict(name="gemm 1000x776x1030", op="gemm", m=1000, n=776, k=1030, b="rows", out="f32"),
        # a training batch through a projection
        dict(name="gemm 8192x8192x4096", op="gemm", m=8192, n=8192, k=4096, b="blocks", out="bf16"),
        # one step of serving 16 sequences: few rows for each expert
        dict(name="experts 16 tokens", op="experts", tokens=16, top=8, experts=64, n=4096, k=2048),
        # a prompt, or a training batch
        dict(name="experts 8192 tokens", op="experts", tokens=8192, top=8, experts=64, n=4096, k=2048),
        # weight gradients of a training batch
        dict(name="wgrad 8192 tokens", op="wgrad", tokens=8192, top=4, experts=32, n=2048, k=1024),
        # serving 16 sequences: order and rows, no padding between the experts
        dict(name="route 16 tokens", op="route", tokens=16, top=8, experts=64, h=4096, align=1, rows="bf16"),
        # a training batch, quantised on the way, each expert's rows padded to whole groups
        dict(name="route 16384 tokens fp8", op="route", tokens=16384, top=8, experts=64, h=4096, align=128, rows="fp8"),
        # serving 16 sequences
        dict(name="combine 16 tokens", op="combine", tokens=16, top=8, experts=64, h=4096, align=1, train=False),
        # a training batch, forward and backward
        dict(name="combine 8191 tokens train", op="combine", tokens=8191, top=6, experts=64, h=4096, align=128, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A matrix width: mostly whole groups, now and then an odd one."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(128, (v + 64) // 128 * 128)


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "experts", "experts", "wgrad", "route", "combine"])
    if op == "quantize":
        along = rng.choice(["rows", "columns", "blocks"])
        return dict(op=op, along=along, rows=_log(rng, 1, 16384), cols=_width(rng, 96, 4096))
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 8192), n=_width(rng, 96, 8192), k=_width(rng, 96, 4096),
                    b=rng.choice(["blocks", "rows"]), out=rng.choice(["bf16", "f32"]))
    experts = rng.choice([8, 16, 32, 60, 64])
    top = rng.randint(1, 8)
    if op == "experts":
        return dict(op=op, tokens=_log(rng, 1, 8192), top=top, experts=experts, n=_width(rng, 96, 4096),
                    k=_width(rng, 96, 2048))
    if op == "wgrad":
        return dict(op=op, tokens=_log(rng, 1, 8192), top=min(top, 4), experts=min(experts, 32), n=_width(rng, 96, 2048),
                    k=_width(rng, 96, 1024))
    h = _width(rng, 96, 4096)
    if op == "route":
        rows = rng.choice(["bf16", "fp8"])
        return dict(op=op, tokens=_log(rng, 1, 16384), top=top, experts=experts, h=h, align=rng.choice([1, 128]), rows=rows)
    return dict(op=op, tokens=_log(rng, 1, 8191), top=min(top, 6), experts=experts, h=h, align=rng.choice([1, 128]),
                train=rng.random() < 0.5)


def _ceil(a, b):
    return -(-a // b)


def _capacity(case):
    """Rows of the sorted layout: every slot, and the most that padding can add."""
    slots, align = case["tokens"] * case["top"], case.get("align", 128 if case["op"] == "wgrad" else 1)
    return (slots + min(case["experts"], slots) * (align - 1)) // align * align


def work(case):
    op = case["op"]
    if op == "quantize":
        n, c = case["rows"] * case["cols"], case["cols"]
        groups = {"rows": case["rows"] * _ceil(c, GROUP), "columns": c * _ceil(case["rows"], GROUP),
                  "blocks": _ceil(case["rows"], GROUP) * _ceil(c, GROUP)}[case["along"]]
        return {"bytes": 3 * n + 4 * groups, "flops": 3 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _ceil(k, GROUP)
        scales = 4 * kb * (m + (n if case["b"] == "rows" else _ceil(n, GROUP)))
        return {"bytes": (m + n) * k + scales + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    slots, e = case["tokens"] * case["top"], case["experts"]
    hit = e * (1 - (1 - case["top"] / e) ** case["tokens"])    # experts that get a token, routed evenly
    if op == "experts":
        n, k = case["n"], case["k"]
        weights = hit * (n * k + 4 * _ceil(n, GROUP) * _ceil(k, GROUP))
        return {"bytes": weights + slots * (k + 4 * _ceil(k, GROUP) + 2 * n), "flops": 2 * slots * n * k}
    if op == "wgrad":
        n, k = case["n"], case["k"]
        return {"bytes": slots * (n + k) * (1 + 4 / GROUP) + 4 * e * n * k, "flops": 2 * slots * n * k}
    h, r = case["h"], _capacity(case)
    if op == "route":
        order = slots * 8 + (slots + r + e + 1) * 4
        row = 2 * h if case["rows"] == "bf16" else h + 4 * _ceil(h, GROUP)
        return {"bytes": order + 2 * case["tokens"] * h + r * row, "flops": 3 * slots * h}
    forward = 2 * slots * h + 8 * slots + 2 * case["tokens"] * h
    if not case["train"]:
        return {"bytes": forward, "flops": 2 * slots * h}
    # forward, then the outputs' gradient and the rows again, the rows' gradient and the weights'
    return {"bytes": forward + 2 * case["tokens"] * h + 2 * slots * h + 2 * r * h + 8 * slots, "flops": 5 * slots * h}


# ------------------------------------------------------------------------------ plain forms

def _groups(x):
    """x (..., C) in groups of 128 along its last axis, zeros behind the end: (..., groups, 128)."""
    pad = -x.shape[-1] % GROUP
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    return x.reshape(*x.shape[:-1], -1, GROUP)


def _quantize_rows(x):
    g = _groups(x.float())
    scale = (g.abs().amax(-1) / TOP).clamp_min(TINY)
    data = (g * (1.0 / scale).unsqueeze(-1)).to(F8).reshape(*x.shape[:-1], -1)
    return data[..., : x.shape[-1]], scale


def _quantize_blocks(x):
    rows, cols = x.shape[-2:]
    x = torch.nn.functional.pad(x.float(), (0, -cols % GROUP, 0, -rows % GROUP))
    g = x.reshape(*x.shape[:-2], x.shape[-2] // GROUP, GROUP, x.shape[-1] // GROUP, GROUP)
    scale = (g.abs().amax((-3, -1)) / TOP).clamp_min(TINY)
    data = (g * (1.0 / scale)[..., :, None, :, None]).to(F8).reshape(x.shape)
    return data[..., :rows, :cols], scale


def _values(data, scale):
    """The fp32 values that e4m3 data stand for: a scale for each 128 along the last axis, and for
    each row or each 128 rows."""
    rows, cols = data.shape[-2:]
    scale = scale.float()
    if scale.shape[-2] != rows:
        scale = scale.repeat_interleave(GROUP, -2)[..., :rows, :]
    return data.float() * scale.repeat_interleave(GROUP, -1)[..., :cols]


def _order(ids, experts, align, capacity):
    flat = ids.reshape(-1)
    hot = (torch.arange(experts, device=ids.device)[:, None] == flat).to(torch.int32)
    before = hot.cumsum(1, dtype=torch.int32)
    counts = before[:, -1]
    length = (counts + align - 1) // align * align
    offsets = torch.nn.functional.pad(length.cumsum(0, dtype=torch.int32), (1, 0))
    kept = (flat >= 0) & (flat < experts)
    place = offsets[flat.clamp(0, experts - 1)] + ((before - hot) * hot).sum(0, dtype=torch.int32)
    position = torch.where(kept, place, -1).to(torch.int32)
    source = torch.full((capacity + 1,), -1, dtype=torch.int32, device=ids.device)
    source[torch.where(kept, place, capacity).long()] = torch.arange(flat.numel(), dtype=torch.int32, device=ids.device)
    return offsets, position.reshape(ids.shape), source[:capacity].contiguous()


def _rows_of(x, source, top):
    """The tokens' rows in sorted order; zeros where a row of the layout has no token."""
    taken = x[(source.clamp_min(0) // top).long()]
    return torch.where((source >= 0)[:, None], taken, torch.zeros((), dtype=x.dtype, device=x.device))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        x = s["x"]
        return {"rows": lambda: _quantize_rows(x), "columns": lambda: _quantize_rows(x.t()),
                "blocks": lambda: _quantize_blocks(x)}[c["along"]]()
    if op == "gemm":
        out = _values(s["a"], s["sa"]) @ _values(s["b"], s["sb"]).t()
        return out if c["out"] == "f32" else out.to(torch.bfloat16)
    if op == "experts":
        # one product for each expert that has rows (fewer operations than padding all of them to the longest)
        a, out = _values(s["a"], s["sa"]), torch.empty(s["a"].shape[0], c["n"], dtype=torch.bfloat16, device="cuda")
        for e, (i, j) in enumerate(zip(s["ends"], s["ends"][1:])):
            if j > i:
                out[i:j] = a[i:j] @ _values(s["b"][e], s["sb"][e]).t()
        out[s["ends"][-1]:] = 0
        return out
    if op == "wgrad":
        a, b = _values(s["a"], s["sa"]), _values(s["b"], s["sb"])
        out = torch.empty(c["experts"], c["n"], c["k"], device="cuda")
        for e, (i, j) in enumerate(zip(s["ends"], s["ends"][1:])):
            torch.matmul(a[:, i:j], b[:, i:j].t(), out=out[e])
        return out
    if op == "route":
        offsets, position, source = _order(s["ids"], c["experts"], c["align"], _capacity(c))
        rows = _rows_of(s["x"], source, c["top"])
        return (offsets, position, source) + (tuple(_quantize_rows(rows)) if c["rows"] == "fp8" else (rows,))
    offsets, position, source = s["order"]
    kept = (position >= 0)[..., None]
    rows = torch.where(kept, s["y"][position.clamp_min(0).long()].float(), torch.zeros((), device=position.device))
    weights = s["weights"][..., None]
    out = (rows * weights).sum(1).to(torch.bfloat16)
    if not c["train"]:
        return out
    grad = s["grad"].float()
    d_weights = (rows * grad[:, None]).sum(-1)
    token = source.clamp_min(0).long()
    d_rows = grad[token // c["top"]] * s["weights"].reshape(-1)[token][:, None] * (source >= 0)[:, None]
    return out, d_rows.to(torch.bfloat16), d_weights


# ------------------------------------------------------------------------------ the package's calls

def _own(s):
    import tensor_core_loop_gb300 as tcl
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return tcl.quantize_fp8(s["x"], along=c["along"])
    if op == "gemm":
        return tcl.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16)
    if op == "experts":
        return tcl.gemm_fp8_experts(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=torch.bfloat16)
    if op == "wgrad":
        return tcl.gemm_fp8_experts_wgrad(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=torch.float32)
    if op == "route":
        order = tcl.sort_by_expert(s["ids"], c["experts"], align=c["align"])
        rows = tcl.quantize_fp8(s["x"], along="rows", order=order) if c["rows"] == "fp8" else (tcl.gather_rows(s["x"], order),)
        return tuple(order) + tuple(rows)
    order = tcl.ExpertOrder(*s["order"])
    out = tcl.combine(s["y"], s["weights"], order)
    if not c["train"]:
        return out
    return (out,) + tuple(tcl.combine_grad(s["grad"], s["y"], s["weights"], order))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------ inputs

def _activations(gen, rows, cols):
    """Hidden states: near normal, a few channels ten times as large."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    loud = torch.rand(cols, device="cuda", generator=gen) < 0.01
    return (x * torch.where(loud, 10.0, 1.0)).to(torch.bfloat16)


def _pitched(data):
    """e4m3 rows at a pitch of whole 16-byte pieces, as a quantising call lays them out."""
    cols = data.shape[-1]
    full = torch.zeros(*data.shape[:-1], _ceil(cols, 16) * 16, dtype=torch.uint8, device=data.device)
    full[..., :cols] = data.contiguous().view(torch.uint8)
    return full.view(F8)[..., :cols]


def _operand(x, blocks=False):
    data, scale = _quantize_blocks(x) if blocks else _quantize_rows(x)
    return _pitched(data), scale if blocks else scale.t().contiguous().t()


def _routing(gen, case):
    """The router's choices and their weights: some experts liked better than others."""
    logits = torch.randn(case["tokens"], case["experts"], device="cuda", generator=gen)
    logits += 0.7 * torch.randn(case["experts"], device="cuda", generator=gen)
    best, ids = logits.topk(min(case["top"], case["experts"]), -1)
    return ids, torch.softmax(best, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "quantize":
        s["x"] = _activations(gen, case["rows"], case["cols"])
        return s
    if op == "gemm":
        s["a"], s["sa"] = _operand(_activations(gen, case["m"], case["k"]))
        b = torch.randn(case["n"], case["k"], device="cuda", generator=gen) * 0.02
        s["b"], s["sb"] = _operand(b, case["b"] == "blocks")
        return s
    ids, weights = _routing(gen, case)
    if op == "experts":
        offsets, _, source = _order(ids, case["experts"], 1, _capacity(case))
        x = _activations(gen, case["tokens"], case["k"])
        s["a"], s["sa"] = _operand(_rows_of(x, source, case["top"]))
        b = torch.randn(case["experts"], case["n"], case["k"], dtype=torch.bfloat16, device="cuda", generator=gen) * 0.02
        s["b"], s["sb"] = _operand(b, True)
        s["offsets"], s["ends"] = offsets, offsets.tolist()
        return s
    if op == "wgrad":
        offsets, _, source = _order(ids, case["experts"], 128, _capacity(case))
        x = _rows_of(_activations(gen, case["tokens"], case["k"]), source, case["top"])
        dy = _rows_of(_activations(gen, case["tokens"], case["n"]), source, case["top"])
        weight = torch.where(source >= 0, weights.reshape(-1)[source.clamp_min(0).long()], 0.0)
        s["a"], s["sa"] = _operand((dy * weight[:, None]).to(torch.bfloat16).t())
        s["b"], s["sb"] = _operand(x.t())
        s["offsets"], s["ends"] = offsets, offsets.tolist()
        return s
    # a batch is filled up with tokens that go nowhere: their ids are -1
    ids = torch.where(torch.rand(case["tokens"], 1, device="cuda", generator=gen) < 0.03, -1, ids)
    if op == "route":
        s["ids"], s["x"] = ids, _activations(gen, case["tokens"], case["h"])
        return s
    s["order"] = _order(ids, case["experts"], case["align"], _capacity(case))
    s["y"] = _activations(gen, s["order"][2].numel(), case["h"])
    s["weights"] = weights
    s["grad"] = _activations(gen, case["tokens"], case["h"])
    return s


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(v):
    """v in 64 bits rounded to the nearest e4m3 value, ties to even; |v| is at most 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-5) - 4)
    return torch.round(v / step) * step


def _exact_quantize(x, along_rows):
    x = x.double()
    rows, cols = x.shape
    r = 1 if along_rows else GROUP
    full = torch.zeros(_ceil(rows, r) * r, _ceil(cols, GROUP) * GROUP, dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x
    tiles = full.unfold(0, r, r).unfold(1, GROUP, GROUP)
    scale = torch.clamp(tiles.abs().flatten(2).max(2).values / 448, min=2.0 ** -126)
    wide = torch.kron(scale, torch.ones(r, GROUP, dtype=torch.float64, device=x.device))
    return _e4m3(full / wide)[:rows, :cols].contiguous(), scale


def _exact_values(data, scale):
    r = 1 if scale.shape[0] == data.shape[0] else GROUP
    wide = torch.kron(scale.double().contiguous(), torch.ones(r, GROUP, dtype=torch.float64, device=data.device))
    return data.double() * wide[: data.shape[0], : data.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["x"].t() if case["along"] == "columns" else s["x"], case["along"] != "blocks")
    if op == "gemm":
        return _exact_values(s["a"], s["sa"]) @ _exact_values(s["b"], s["sb"]).T
    if op in ("experts", "wgrad"):
        ends = s["ends"]
        a = _exact_values(s["a"], s["sa"])
        if op == "wgrad":
            b = _exact_values(s["b"], s["sb"])
            return torch.stack([a[:, i:j] @ b[:, i:j].T for i, j in zip(ends, ends[1:])])
        out = torch.zeros(a.shape[0], case["n"], dtype=torch.float64, device=a.device)
        for e, (i, j) in enumerate(zip(ends, ends[1:])):
            out[i:j] = a[i:j] @ _exact_values(s["b"][e], s["sb"][e]).T
        return out
    if op == "route":
        # the places, token by token in the order of their slots
        align, cap = case["align"], _capacity(case)
        ids = s["ids"].reshape(-1).cpu()
        by = torch.argsort(torch.where(ids >= 0, ids, case["experts"]), stable=True)
        source, at = torch.full((cap,), -1, dtype=torch.int64), 0
        for e in range(case["experts"]):
            mine = by[ids[by] == e]
            source[at:at + len(mine)] = mine
            at += _ceil(len(mine), align) * align
        source = source.cuda()
        rows = s["x"].double()[source.clamp_min(0) // case["top"]]
        rows[source < 0] = 0
        if case["rows"] == "bf16":
            return None, None, None, rows
        return (None, None, None) + _exact_quantize(rows, True)
    position, source = s["order"][1].long(), s["order"][2].long()
    out = torch.zeros(case["tokens"], case["h"], dtype=torch.float64, device="cuda")
    d_weights = torch.zeros(position.shape, dtype=torch.float64, device="cuda")
    d_rows = torch.zeros(source.numel(), case["h"], dtype=torch.float64, device="cuda")
    grad = s["grad"].double()
    for j in range(position.shape[1]):
        t = torch.nonzero(position[:, j] >= 0).flatten()
        row = position[t, j]
        y, w = s["y"][row].double(), s["weights"][t, j].double()[:, None]
        out[t] += w * y
        d_weights[t, j] = (grad[t] * y).sum(1)
        d_rows[row] = w * grad[t]
    return (out, d_rows, d_weights) if case["train"] else out
