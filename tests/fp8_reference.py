"""The e4m3 operators and the expert routing in 64 bits (NumPy and PyTorch on the CPU), written
from the definitions in include/tcl_fp8.h; shares no code with the library.

Bounds, for S = sum over k of |a·b| with the scales applied, G groups of 128 along K:
a group's sum on the tensor core takes at most 128 fp32 additions of exact products, each
rounded or truncated, so off by at most 2^-23 of a magnitude at most the group's S; the scales'
product and the addition into the running sum are three roundings for each group, and the running
sum takes G additions. Together at most (128 + 3 + G)·2^-23·S, and a bf16 result is off by at most
2^-8 of its own magnitude more (bf16 keeps 8 bits; half of 2^-133 where it is subnormal)."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 128


def groups(n: int) -> int:
    return -(-n // GROUP)


def widen(scale, shape):
    """Scales of every row or of every 128 rows, one for each value of a matrix of `shape`."""
    s = scale.double()
    if s.shape[-2] != shape[-2]:
        s = s.repeat_interleave(GROUP, -2)[..., : shape[-2], :]
    return s.repeat_interleave(GROUP, -1)[..., : shape[-1]]


def values(data, scale):
    return data.cpu().double() * widen(scale.cpu(), data.shape)


def product_bound(a, b, out_dtype):
    """(C, bound) for values a (M x K) and b (N x K) in 64 bits."""
    ref = a @ b.t()
    bound = (GROUP + 3 + groups(a.shape[1])) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound) + 2.0 ** -134
    return ref, bound + 2.0 ** -149


def check(got, ref, bound, what=""):
    got = got.cpu().double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {int((over > 0).sum())} of {over.numel()} outside, worst by {float(over.max()):.3g}"


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, of numbers of magnitude at most 448·(1 + 2^-20)."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.clip(np.rint(v / step) * step, -448, 448)


def quantize(x: torch.Tensor, rows_per_group: int):
    """(values of the data, scales) by the definition's fp32 steps, for finite x (rows x cols)."""
    x = x.cpu().float().numpy()
    r, c = x.shape
    rg = rows_per_group
    full = np.zeros((-(-r // rg) * rg, groups(c) * GROUP), np.float32)
    full[:r, :c] = x
    t = np.abs(full).reshape(full.shape[0] // rg, rg, groups(c), GROUP).max((1, 3))
    s = np.maximum(t / np.float32(448), np.float32(2.0 ** -126)).astype(np.float32)
    inv = (np.float32(1) / s).astype(np.float32)
    wide = np.repeat(np.repeat(inv, rg, 0), GROUP, 1)
    with np.errstate(over="ignore"):
        q = e4m3((full * wide).astype(np.float32).astype(np.float64))
    return torch.from_numpy(q[:r, :c]), torch.from_numpy(s)


def order(ids, experts: int, align: int, rows: int):
    """offsets, position, source as lists, slot by slot."""
    flat = ids.reshape(-1).tolist()
    of = [[i for i, e in enumerate(flat) if e == x] for x in range(experts)]
    offsets, position, source = [0], [-1] * len(flat), [-1] * rows
    for mine in of:
        for k, i in enumerate(mine):
            position[i] = offsets[-1] + k
            source[offsets[-1] + k] = i
        offsets.append(offsets[-1] + -(-len(mine) // align) * align)
    return offsets, position, source
