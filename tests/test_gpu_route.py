"""Sorting tokens by expert, gathering and combining their rows, and the gradients, on the GPU."""
from __future__ import annotations

import pytest
import torch

import fp8_reference as ref
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


def make_ids(tokens, top, experts, seed, dtype=torch.int64, lo=-1):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, experts, (tokens, top), generator=g).to(dtype)


SORTS = [(0, 2, 4, 1), (0, 2, 4, 128), (1, 1, 1, 1), (1, 8, 64, 1), (16, 8, 64, 1), (16, 8, 64, 128), (100, 3, 7, 5), (513, 8, 60, 128),
         (512, 8, 256, 1), (1024, 4, 33, 16), (5000, 3, 1024, 1), (3000, 7, 128, 128), (20000, 2, 5, 64)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top,experts,align", SORTS)
def test_sort(tokens, top, experts, align, dtype):
    ids = make_ids(tokens, top, experts, tokens + top, dtype)
    got = tcl.sort_by_expert(ids.to(DEV), experts, align=align)
    offsets, position, source = ref.order(ids, experts, align, got.source.numel())
    assert got.offsets.tolist() == offsets
    assert got.position.reshape(-1).tolist() == position
    assert got.source.tolist() == source
    assert offsets[-1] <= got.source.numel()


@pytest.mark.parametrize("tokens", [10, 6000])
def test_sort_one_expert_none_and_wild_ids(tokens):
    for ids in (torch.full((tokens, 2), 3), torch.full((tokens, 2), -1), torch.full((tokens, 2), 2 ** 40 + 1),
                torch.full((tokens, 2), 8), torch.arange(2 * tokens).flip(0).view(tokens, 2) % 11 - 2):
        got = tcl.sort_by_expert(ids.to(DEV), 8, align=128)
        offsets, position, source = ref.order(ids, 8, 128, got.source.numel())
        assert got.offsets.tolist() == offsets
        assert got.position.reshape(-1).tolist() == position and got.source.tolist() == source


CASES = [(1, 1, 1, 1, 1), (1, 8, 64, 1, 4096), (16, 8, 64, 1, 1000), (33, 3, 5, 16, 257), (200, 6, 9, 128, 512), (70, 9, 20, 1, 2056),
         (40, 17, 30, 8, 24)]


def setup(tokens, top, experts, align, cols, dtype):
    g = torch.Generator().manual_seed(tokens + cols)
    ids = make_ids(tokens, top, experts, 3)
    if tokens > 1:
        ids[0] = -1                       # a token that goes nowhere
    order = tcl.sort_by_expert(ids.to(DEV), experts, align=align)
    rows = order.source.numel()
    x = torch.randn(tokens, cols, generator=g).to(dtype)
    y = torch.randn(rows, cols, generator=g).to(dtype)
    grad = torch.randn(tokens, cols, generator=g).to(dtype)
    w = torch.rand(tokens, top, generator=g)
    return order, x, y, grad, w


def combine_bound(terms, dtype):
    """Each of the sum's terms and additions rounded in fp32, the result to its type."""
    n = terms.shape[1]
    b = (n + 1) * 2.0 ** -24 * terms.abs().sum(1)
    return b + (2.0 ** -8 * (terms.sum(1).abs() + b) if dtype == BF16 else 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,top,experts,align,cols", CASES)
def test_gather_combine_and_gradients(tokens, top, experts, align, cols, dtype):
    order, x, y, grad, w = setup(tokens, top, experts, align, cols, dtype)
    source, position = order.source.cpu().long(), order.position.cpu().long()
    rows = tcl.gather_rows(x.to(DEV), order).cpu()
    assert torch.equal(rows, torch.where((source >= 0)[:, None], x[source.clamp_min(0) // top], torch.zeros((), dtype=dtype)))

    kept = (position >= 0)[..., None]
    picked = torch.where(kept, y.double()[position.clamp_min(0)], torch.zeros((), dtype=torch.float64))
    for weights in (w, None):
        terms = picked * (w.double()[..., None] if weights is not None else 1.0)
        out = tcl.combine(y.to(DEV), weights.to(DEV) if weights is not None else None, order).cpu().double()
        assert bool(((out - terms.sum(1)).abs() <= combine_bound(terms, dtype)).all())

        dy, dw = tcl.combine_grad(grad.to(DEV), y.to(DEV), weights.to(DEV) if weights is not None else None, order)
        slot = source.clamp_min(0)
        f = (w.double().reshape(-1)[slot] if weights is not None else torch.ones(len(slot)).double()) * (source >= 0)
        want = f[:, None] * grad.double()[slot // top]
        half = 2.0 ** -8 if dtype == BF16 else 0.0
        assert bool(((dy.cpu().double() - want).abs() <= want.abs() * (half + 2.0 ** -24 + half * 2.0 ** -24)).all())
        prods = picked * grad.double()[:, None]
        # a thread adds 8 columns of every 2,048, then 5 + 8 additions join the threads
        adds = 8 * -(-cols // 2048) + 13 + 1
        assert bool(((dw.cpu().double() - prods.sum(-1)).abs() <= adds * 2.0 ** -24 * prods.abs().sum(-1)).all())
        assert bool((dw.cpu()[position < 0] == 0).all())


def test_gradients_against_differences():
    """combine is linear in the rows and in the weights: central differences in 64 bits are exact."""
    order, x, y, grad, w = setup(40, 4, 6, 8, 96, F32)
    position, top = order.position.cpu().long(), 4
    dy, dw = tcl.combine_grad(grad.to(DEV), y.to(DEV), w.to(DEV), order)
    g = torch.Generator().manual_seed(9)

    def loss(rows, weights):
        picked = torch.where((position >= 0)[..., None], rows[position.clamp_min(0)], torch.zeros((), dtype=torch.float64))
        return float(((picked * weights[..., None]).sum(1) * grad.double()).sum())

    for _ in range(4):
        d = torch.randn(y.shape, generator=g).double()
        slope = (loss(y.double() + d, w.double()) - loss(y.double() - d, w.double())) / 2
        prods = dy.cpu().double() * d
        assert abs(float(prods.sum()) - slope) <= 1e-6 * float(prods.abs().sum())
        d = torch.randn(w.shape, generator=g).double()
        slope = (loss(y.double(), w.double() + d) - loss(y.double(), w.double() - d)) / 2
        prods = dw.cpu().double() * d
        assert abs(float(prods.sum()) - slope) <= 1e-5 * float(prods.abs().sum())
    # the gradient of gather_rows: sum of x's rows times any row gradient
    dr = torch.randn(y.shape, generator=g)
    dx = tcl.combine(dr.to(DEV), None, order).cpu().double()
    d = torch.randn(x.shape, generator=g).double()
    source = order.source.cpu().long()
    slope = float((torch.where((source >= 0)[:, None], d[source.clamp_min(0) // top], torch.zeros((), dtype=torch.float64)) * dr.double()).sum())
    assert abs(float((dx * d).sum()) - slope) <= 1e-6 * float((dx * d).abs().sum()) + 1e-6 * abs(slope)


def test_strides_and_alignment():
    order, x, y, grad, w = setup(20, 3, 4, 1, 100, BF16)
    want_rows = tcl.gather_rows(x.to(DEV), order)
    want_out = tcl.combine(y.to(DEV), w.to(DEV), order)
    want_dy, want_dw = tcl.combine_grad(grad.to(DEV), y.to(DEV), w.to(DEV), order)
    for off, pitch in ((0, 120), (1, 113), (8, 112)):
        def wide(t):
            big = torch.full((t.shape[0], pitch + off), float("nan"), dtype=t.dtype, device=DEV)
            big[:, off:off + t.shape[1]] = t.to(DEV)
            return big[:, off:off + t.shape[1]]
        assert torch.equal(tcl.gather_rows(wide(x), order), want_rows)
        assert torch.equal(tcl.combine(wide(y), w.to(DEV), order), want_out)
        dy, dw = tcl.combine_grad(wide(grad), wide(y), w.to(DEV), order)
        assert torch.equal(dy, want_dy) and torch.equal(dw, want_dw)


def test_non_finite_rows_reach_only_their_token():
    order, x, y, grad, w = setup(20, 3, 4, 16, 64, F32)
    source = order.source.cpu()
    y[source < 0] = float("nan")          # rows without a slot are never read
    row = int(torch.nonzero(source >= 0)[0])
    y[row, 5] = float("inf")
    out = tcl.combine(y.to(DEV), w.to(DEV), order).cpu()
    bad = ~torch.isfinite(out)
    assert bad.sum() == 1 and bool(bad[int(source[row]) // 3, 5])
    _, dw = tcl.combine_grad(grad.to(DEV), y.to(DEV), w.to(DEV), order)
    assert int((~torch.isfinite(dw)).sum()) == 1


def test_no_tokens():
    order = tcl.sort_by_expert(torch.empty(0, 3, dtype=torch.int64, device=DEV), 4)
    assert order.offsets.tolist() == [0] * 5 and order.source.numel() == 0
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    assert tcl.gather_rows(x, order).shape == (0, 64) and tcl.combine(x, None, order).shape == (0, 64)
    assert tcl.quantize_fp8(x, order=order)[0].shape == (0, 64)
    dy, dw = tcl.combine_grad(x, x, None, order)
    assert dy.shape == (0, 64) and dw.shape == (0, 3)


def test_past_32_bit_offsets():
    rows, cols = 530_000, 4096           # 2.17e9 elements
    ids = torch.arange(rows, device=DEV).remainder(2).view(-1, 1)
    order = tcl.sort_by_expert(ids, 2)
    x = torch.arange(rows, device=DEV).remainder(251).to(BF16)[:, None].expand(rows, cols).contiguous()
    y = tcl.gather_rows(x, order)
    half = rows // 2
    assert torch.equal(y[half:], x[1::2]) and torch.equal(y[:half], x[::2])
    del x
    back = tcl.combine(y, None, order)
    assert torch.equal(back[-1000:, 0].float(), torch.arange(rows - 1000, rows, device=DEV).remainder(251).float())
    assert torch.equal(back[:, 0], back[:, -1])
    del y, back


def test_graph():
    ids = make_ids(300, 4, 16, 1).to(DEV)
    x = torch.randn(300, 256, device=DEV).to(BF16)

    def step():
        order = tcl.sort_by_expert(ids, 16, align=128)
        return order.source, tcl.gather_rows(x, order), *tcl.quantize_fp8(x, order=order)

    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    ids.copy_(make_ids(300, 4, 16, 2))
    want = step()
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u.float(), v.float())
