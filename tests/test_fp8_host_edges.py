"""Edges of the fp8 and routing entry points on the host (no GPU): sizes at the end of 32 bits, and what
a call on a given stream does with its operands."""
from __future__ import annotations

from contextlib import nullcontext

import pytest
import torch

import tensor_core_loop_gb300 as tcl
from tensor_core_loop_gb300 import fp8
from test_fp8_host import L, P, experts, gemm, wgrad  # noqa: F401

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("size", [TOP, TOP - 65_535])
def test_sizes_at_the_end_of_32_bits_are_refused(L, size):  # noqa: F811
    """Index arithmetic in 32 bits rounds sizes up to whole tiles: it needs room above them."""
    for kw in (dict(M=size), dict(N=size, ldc=TOP), dict(K=size, lda=TOP, ldb=TOP)):
        assert gemm(L, **kw) == 2, kw
    for kw in (dict(rows=size), dict(N=size, ldc=TOP, be=2 ** 40), dict(K=size, lda=TOP, ldb=TOP, be=2 ** 40)):
        assert experts(L, **kw) == 2, kw
    for kw in (dict(rows=size, lda=TOP, ldb=TOP), dict(N=size, ce=2 ** 40), dict(K=size, ldc=TOP, ce=2 ** 40)):
        assert wgrad(L, **kw) == 2, kw
    big = TOP
    rows, cols, blocks = L.tcl_quantize_fp8_rows, L.tcl_quantize_fp8_columns, L.tcl_quantize_fp8_blocks
    assert rows(0, size, 64, P, 64, None, 1, None, 0, P, 64, P, 1, 4, None) == 2
    assert rows(0, 4, size, P, big, None, 1, None, 0, P, big, P, 1, 4, None) == 2
    assert rows(0, 4, 64, P, 64, P, 1, P, size, P, 64, P, 1, 4, None) == 2
    assert cols(0, size, 64, P, 64, None, 1, 0, P, big, P, 1, 64, None) == 2
    assert cols(0, 4, size, P, big, None, 1, 0, P, 64, P, 1, 64, None) == 2
    assert cols(0, 4, 64, P, 64, P, 1, size, P, big, P, 1, 64, None) == 2
    assert blocks(0, 1, size, 64, P, 64, 0, 0, P, 64, 0, P, None) == 2
    assert blocks(0, 1, 4, size, P, big, 0, 0, P, big, 0, P, None) == 2
    assert L.tcl_sort_by_expert(size, 1, P, 4, 4, 1, TOP, P, P, P, None) == 2
    assert L.tcl_sort_by_expert(4, 1, P, 4, 4, 1, size, P, P, P, None) == 2
    for tokens, n, width in ((size, 8, 64), (4, size, 64), (4, 8, size)):
        assert L.tcl_gather_rows(0, tokens, 2, n, width, P, big, P, P, P, big, None) == 2
        assert L.tcl_combine(0, tokens, 2, n, width, P, big, P, P, P, big, None) == 2
        assert L.tcl_combine_grad(0, tokens, 2, n, width, P, big, P, big, P, P, P, P, big, P, None) == 2


def meta(shape, stride, dtype):
    return torch.empty_strided(shape, stride, dtype=dtype, device="meta")


def test_numbers_past_32_bits_are_refused_not_cut_off():
    """A leading dimension or a count beyond the C interface's ints (ctypes keeps the low 32 bits)."""
    far = 2 ** 32 + 64
    bf16, f8, f32, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
    x, long = meta((2, 64), (far, 1), bf16), meta((far, 64), (64, 1), bf16)
    a, s = meta((2, 64), (far, 1), f8), meta((2, 1), (1, 2), f32)
    b, bs = meta((64, 64), (64, 1), f8), meta((64, 1), (1, 64), f32)
    w, ws, off = meta((3, 64, 64), (4096, 64, 1), f8), meta((3, 64, 1), (64, 1, 64), f32), meta((4,), (1,), i32)
    out = meta((64, 64), (far, 1), bf16)
    order = tcl.ExpertOrder(off, meta((2, 1), (1, 1), i32), meta((2,), (1,), i32))
    wide = tcl.ExpertOrder(off, meta((2, 2 ** 31), (2 ** 31, 1), i32), meta((2,), (1,), i32))
    many = tcl.ExpertOrder(off, meta((2, 1), (1, 1), i32), meta((far,), (1,), i32))
    y = meta((2, 64), (64, 1), bf16)
    for call in (
        lambda: tcl.quantize_fp8(x),
        lambda: tcl.quantize_fp8(x, along="columns"),
        lambda: tcl.quantize_fp8(long, along="blocks"),
        lambda: tcl.quantize_fp8(meta((far, 2, 64), (128, 64, 1), bf16), along="blocks"),
        lambda: tcl.quantize_fp8(meta((2, far), (far, 1), bf16)),
        lambda: tcl.quantize_fp8(y, order=many),
        lambda: tcl.quantize_fp8(y, order=wide),
        lambda: tcl.gemm_fp8(a, s, b, bs),
        lambda: tcl.gemm_fp8(b, bs, b, bs, out=out),
        lambda: tcl.gemm_fp8_experts(a, s, w, ws, off),
        lambda: tcl.gemm_fp8_experts(b, bs, meta((far, 64, 64), (4096, 64, 1), f8), meta((far, 64, 1), (64, 1, 64), f32),
                                     meta((far + 1,), (1,), i32)),
        lambda: tcl.gemm_fp8_experts_wgrad(a, s, b, bs, off),
        lambda: tcl.sort_by_expert(meta((far, 1), (1, 1), torch.int64), 4),
        lambda: tcl.sort_by_expert(meta((4, far), (far, 1), torch.int64), 4),
        lambda: tcl.gather_rows(x, order),
        lambda: tcl.combine(x, None, order),
        lambda: tcl.combine_grad(x, y, None, order),
    ):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_operands_are_recorded_on_the_given_stream(monkeypatch):
    """The caching allocator must know that the given stream reads them (it would hand their memory out
    again once the caller drops them)."""
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(fp8, "_on", lambda stream: nullcontext())
    monkeypatch.setattr(fp8, "_call", lambda *args: None)
    bf16, f8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    stream = object()
    x = torch.zeros(4, 64, dtype=bf16)
    a, s = torch.zeros(128, 128, dtype=f8), torch.zeros(128, 1)
    w, ws = torch.zeros(2, 128, 128, dtype=f8), torch.zeros(2, 1, 1)
    off, ids = torch.zeros(3, dtype=i32), torch.zeros(4, 2, dtype=torch.int64)
    pos, src, weights = torch.zeros(4, 2, dtype=i32), torch.zeros(8, dtype=i32), torch.zeros(4, 2)
    y, out = torch.zeros(8, 64, dtype=bf16), torch.zeros(128, 128, dtype=bf16)
    dw = torch.zeros(2, 128, 128, dtype=bf16)
    order = tcl.ExpertOrder(off, pos, src)
    for call, tensors in (
        (lambda st: tcl.quantize_fp8(x, stream=st), [x]),
        (lambda st: tcl.quantize_fp8(x, order=order, stream=st), [x, pos, src]),
        (lambda st: tcl.quantize_fp8(x, along="columns", order=order, stream=st), [x, pos, src]),
        (lambda st: tcl.quantize_fp8(x, along="blocks", stream=st), [x]),
        (lambda st: tcl.gemm_fp8(a, s, a, s, out=out, stream=st), [a, s, out]),
        (lambda st: tcl.gemm_fp8_experts(a, s, w, ws, off, out=out, stream=st), [a, s, w, ws, off, out]),
        (lambda st: tcl.gemm_fp8_experts_wgrad(a, s, a, s, off, out=dw, stream=st), [a, s, off, dw]),
        (lambda st: tcl.sort_by_expert(ids, 2, stream=st), [ids]),
        (lambda st: tcl.gather_rows(x, order, stream=st), [x, pos, src]),
        (lambda st: tcl.combine(y, weights, order, stream=st), [y, weights, pos]),
        (lambda st: tcl.combine_grad(x, y, weights, order, stream=st), [x, y, weights, pos, src]),
    ):
        recorded.clear()
        call(stream)
        assert {p for p, _ in recorded} >= {t.data_ptr() for t in tensors}
        assert all(st is stream for _, st in recorded)
        recorded.clear()
        call(None)
        assert not recorded
