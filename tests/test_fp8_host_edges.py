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
