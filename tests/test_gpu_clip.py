"""The norm over many tensors and their scaling on the GPU, against 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

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


def tensors(seed, sizes, dtypes, scale=1.0, offset=0):
    """`offset`: elements behind an aligned address."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        d = dtypes[i % len(dtypes)]
        room = (torch.randn(n + offset, generator=g, dtype=torch.float64) * scale).to(d).to(DEV)
        out.append(room[offset:])
    return out


def norm_of(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def check(ts, norm, got, bound):
    """32 squares are added in fp32 (32 roundings of half a step each, so half of that in the root), the rest in
    fp64; the result is rounded to fp32, the scaled values to their type after one product with an fp32 factor."""
    want = norm_of(ts)
    assert abs(float(norm) - want) <= 20 * 2.0 ** -24 * want
    f = bound / want if want > bound else 1.0
    for t, g in zip(ts, got):
        assert g.dtype == t.dtype and g.shape == t.shape
        if f == 1.0:
            assert torch.equal(g, t)
            continue
        step = 2.0 ** -8 if t.dtype == BF16 else 2.0 ** -24
        exact = t.double() * f
        assert ((g.double() - exact).abs() <= (step + 24 * 2.0 ** -24) * exact.abs() + 1e-37).all()


@pytest.mark.parametrize("bound", [0.0, 0.7, 1e9])
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (BF16, F32)])
@pytest.mark.parametrize("sizes,offset", [((1,), 0), ((7, 0, 1), 0), ((4096, 4097, 0, 33), 1), ((100003, 5, 65536, 65537), 0),
                                          ((300001,), 3), ((0, 0), 0), (tuple(range(600)), 0), ((5_000_001, 3_000_000), 0)])
def test_clip(sizes, offset, dtypes, bound):
    ts = tensors(len(sizes), sizes, dtypes, offset=offset)
    before = [t.clone() for t in ts]
    norm = tcl.grad_norm(ts)
    out = [torch.full_like(t, 5.0) for t in ts]
    again = tcl.clip_grads(ts, bound, out=out)
    assert torch.equal(norm, again)
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    check(before, norm, out, bound)
    inplace = tcl.clip_grads(ts, bound)
    assert torch.equal(inplace, norm) and all(torch.equal(t, o) for t, o in zip(ts, out))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_norm_that_is_not_finite_scales_nothing(dtype, value):
    ts = tensors(3, (1000, 70000), (dtype,))
    ts[1][69990] = value
    out = [torch.zeros_like(t) for t in ts]
    norm = tcl.clip_grads(ts, 1.0, out=out)
    assert math.isnan(float(norm)) if math.isnan(value) else float(norm) == math.inf
    for t, o in zip(ts, out):
        assert torch.equal(t.view(torch.int16 if dtype == BF16 else torch.int32), o.view(torch.int16 if dtype == BF16 else torch.int32))


@pytest.mark.parametrize("scale", [1e-30, 3e-22, 1e20, 3e34])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_past_the_range_of_fp32(dtype, scale):
    ts = tensors(5, (40000, 9, 8192), (dtype,), scale=scale)
    want = norm_of(ts)
    assert abs(float(tcl.grad_norm(ts)) - want) <= 20 * 2.0 ** -24 * want
    bound = want / 3
    out = [torch.zeros_like(t) for t in ts]
    norm = tcl.clip_grads(ts, bound, out=out)
    check(ts, norm, out, float(torch.tensor(bound, dtype=F32)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_norm_past_the_range_of_fp32_scales_nothing(dtype):
    """Finite in 64 bits, but told as infinity."""
    ts = [torch.full((9000,), 2e38, dtype=dtype, device=DEV)]
    out = [torch.zeros_like(ts[0])]
    assert float(tcl.clip_grads(ts, 1.0, out=out)) == math.inf and torch.equal(out[0], ts[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1])
def test_factors_below_the_normal_numbers(dtype, offset):
    """bound/norm of 1e-42 or so: results are normal numbers all the same."""
    ts = tensors(7, (9000, 21), (dtype,), scale=3e35, offset=offset)
    bound = float(torch.tensor(1e-5, dtype=F32))
    out = [torch.zeros(t.numel() + 1, dtype=dtype, device=DEV)[1:] for t in ts]
    check(ts, tcl.clip_grads(ts, bound, out=out), out, bound)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", range(8))
def test_results_at_another_alignment(dtype, shift):
    ts = tensors(6, (70001, 8192, 3), (dtype,), offset=shift)
    for other in (shift, 0, 3):
        out = [torch.zeros(t.numel() + other, dtype=dtype, device=DEV)[other:] for t in ts]
        check(ts, tcl.clip_grads(ts, 2.0, out=out), out, 2.0)


def test_zeros_have_norm_zero():
    ts = [torch.zeros(100000, device=DEV), torch.zeros(3, dtype=BF16, device=DEV)]
    assert float(tcl.clip_grads(ts, 0.0)) == 0.0 and not any(t.any() for t in ts)


def test_results_that_share_memory_are_refused():
    a, b = tensors(8, (4096, 50), (F32,))
    before = a.clone()
    for call in (lambda: tcl.clip_grads([a, b, a], 0.1), lambda: tcl.clip_grads([a, a[4000:]], 0.1),
                 lambda: tcl.clip_grads([b, a[:50]], 0.1, out=[a[10:60], b]), lambda: tcl.clip_grads([b, b + 1], 0.1, out=[a[:50], a[49:99]])):
        with pytest.raises(ValueError, match="shares memory"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(a, before)
    norm = tcl.grad_norm([a, a])   # (reads alone may)
    assert abs(float(norm) - math.sqrt(2) * norm_of([a])) <= 20 * 2.0 ** -24 * float(norm)
