"""The fp8 and routing entry points on the host (no GPU): exports, refusals of the C ABI before it
touches a device, and the binding's checks of its arguments."""
from __future__ import annotations

import os
import re

import pytest
import torch

import fp8_reference as ref
import tensor_core_loop_gb300 as tcl
from tensor_core_loop_gb300 import fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, PO, P2 = 0x10000000, 0x10000001, 0x10000002   # well-formed, odd and 2-byte aligned addresses, never used


@pytest.fixture(scope="module")
def L():
    from tensor_core_loop_gb300 import _build
    _build.build()
    return fp8._lib()


def test_exports(L):
    text = open(os.path.join(ROOT, "include", "tcl_fp8.h")).read()
    declared = set(re.findall(r"TCL_API\s+[\w\s\*]+?\b(\w+)\s*\(", text))
    assert declared == set(tcl.EXPORTED_SYMBOLS_FP8)
    for name in declared:
        assert hasattr(L, name)
    assert f"#define TCL_MAX_EXPERTS {fp8.MAX_EXPERTS}" in text


def gemm(L, **kw):
    d = dict(M=4, N=64, K=64, A=P, lda=64, SA=P, sar=1, sag=4, B=P, ldb=64, SB=P, kind=0, sbr=1, sbg=64, C=P, ldc=64, out=1)
    d.update(kw)
    return L.gemm_fp8(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(A=0), 1), (dict(SA=0), 1), (dict(B=0), 1), (dict(SB=0), 1),
    (dict(C=0), 1), (dict(lda=63), 3), (dict(ldb=63), 3), (dict(ldc=63), 3), (dict(SA=P2), 4), (dict(SB=P2), 4),
    (dict(C=PO), 4), (dict(C=P2, out=0), 4), (dict(out=2), 8), (dict(kind=2), 8)])
def test_gemm_refuses(L, kw, status):
    assert gemm(L, **kw) == status


def experts(L, **kw):
    d = dict(rows=4, E=2, N=64, K=64, A=P, lda=64, SA=P, sar=1, sag=4, B=P, ldb=64, be=4096, SB=P, kind=1, sbe=1, sbr=1, sbg=1,
             off=P, C=P, ldc=64, out=1)
    d.update(kw)
    return L.gemm_fp8_experts(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(E=0), 2), (dict(E=1025), 8), (dict(off=0), 1), (dict(off=P2), 4), (dict(be=4095), 3),
    (dict(A=0), 1), (dict(B=0), 1), (dict(C=0), 1), (dict(ldc=1), 3), (dict(out=5), 8), (dict(kind=-1), 8)])
def test_experts_refuse(L, kw, status):
    assert experts(L, **kw) == status


def wgrad(L, **kw):
    d = dict(rows=128, E=2, N=64, K=64, A=P, lda=128, SA=P, sar=1, sag=64, B=P, ldb=128, SB=P, sbr=1, sbg=64, off=P, C=P, ldc=64,
             ce=4096, out=0)
    d.update(kw)
    return L.gemm_fp8_experts_wgrad(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(E=0), 2), (dict(E=2000), 8), (dict(off=0), 1), (dict(C=0), 1),
    (dict(A=0), 1), (dict(SB=0), 1), (dict(lda=127), 3), (dict(ldb=1), 3), (dict(ldc=63), 3), (dict(ce=4095), 3),
    (dict(C=P2), 4), (dict(off=PO), 4), (dict(out=2), 8)])
def test_wgrad_refuses(L, kw, status):
    assert wgrad(L, **kw) == status


def test_quantize_refuses(L):
    def rows(**kw):
        d = dict(t=0, rows=4, cols=64, X=P, ldx=64, pos=None, top=1, src=None, out=0, Q=P, ldq=64, S=P, sr=1, sg=4)
        d.update(kw)
        return L.tcl_quantize_fp8_rows(*d.values(), None)
    assert rows(t=2) == 8 and rows(rows=-1) == 2 and rows(cols=0) == 2 and rows(X=0) == 1 and rows(Q=0) == 1 and rows(S=0) == 1
    assert rows(ldx=63) == 3 and rows(ldq=63) == 3 and rows(X=PO) == 4 and rows(t=1, X=P2) == 4 and rows(S=P2) == 4
    assert rows(pos=P, top=0, src=P, out=4) == 2 and rows(pos=P, out=4) == 1 and rows(pos=P, src=P, out=-1) == 2

    def cols(**kw):
        d = dict(t=0, rows=4, cols=64, X=P, ldx=64, src=None, top=1, out=0, Q=P, ldq=4, S=P, sr=1, sg=4)
        d.update(kw)
        return L.tcl_quantize_fp8_columns(*d.values(), None)
    assert cols(ldq=3) == 3 and cols(src=P, out=5) == 3 and cols(src=P, top=0) == 2 and cols(X=0) == 1 and cols(X=PO) == 4

    def blocks(**kw):
        d = dict(t=0, batch=2, rows=4, cols=64, X=P, ldx=64, xb=256, tr=0, Q=P, ldq=64, qb=256, S=P)
        d.update(kw)
        return L.tcl_quantize_fp8_blocks(*d.values(), None)
    assert blocks(batch=-1) == 2 and blocks(tr=2) == 8 and blocks(qb=255) == 3 and blocks(tr=1, ldq=3) == 3 and blocks(S=0) == 1


def test_routing_refuses(L):
    def sort(**kw):
        d = dict(tokens=4, top=2, ids=P, bytes=8, E=4, align=1, rows=8, off=P, pos=P, src=P)
        d.update(kw)
        return L.tcl_sort_by_expert(*d.values(), None)
    assert sort(bytes=2) == 8 and sort(E=1025) == 8 and sort(align=0) == 8 and sort(align=129) == 8
    assert sort(tokens=-1) == 2 and sort(top=0) == 2 and sort(E=0) == 2 and sort(rows=7) == 2 and sort(align=128, rows=384) == 2
    assert sort(ids=0) == 1 and sort(off=0) == 1 and sort(pos=0) == 1 and sort(src=0) == 1
    assert sort(ids=P2) == 4 and sort(off=P2) == 4
    assert L.tcl_gather_rows(0, 4, 2, 8, 64, P, 63, P, P, P, 64, None) == 3
    assert L.tcl_gather_rows(3, 4, 2, 8, 64, P, 64, P, P, P, 64, None) == 8
    assert L.tcl_gather_rows(0, 4, 2, 8, 64, P, 64, P, None, P, 64, None) == 1
    assert L.tcl_combine(0, 4, 0, 8, 64, P, 64, P, P, P, 64, None) == 2
    assert L.tcl_combine(1, 4, 2, 8, 64, P2, 64, P, P, P, 64, None) == 4
    assert L.tcl_combine(0, 4, 2, 8, 64, P, 64, P, P, P, 1, None) == 3
    assert L.tcl_combine_grad(0, 4, 2, 8, 64, 0, 64, P, 64, P, P, P, P, 64, P, None) == 1
    assert L.tcl_combine_grad(0, 4, 2, 8, 64, P, 64, P, 63, P, P, P, P, 64, P, None) == 3
    assert L.tcl_combine_grad(0, 4, 2, 8, 64, P, 64, P, 64, P, P, None, P, 64, P, None) == 1


def test_binding_refuses():
    f8 = torch.float8_e4m3fn
    a, s = torch.zeros(4, 256, dtype=f8), torch.zeros(4, 2)
    b, bs = torch.zeros(64, 256, dtype=f8), torch.zeros(1, 2)
    off = torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros(2, 64, 256, dtype=f8), torch.zeros(2, 1, 2)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    order = tcl.ExpertOrder(off, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32))
    for err, call in [
        (ValueError, lambda: tcl.gemm_fp8(a, s, b, bs)),                                   # not on a GPU
        (TypeError, lambda: tcl.gemm_fp8(a.float(), s, b, bs)),
        (TypeError, lambda: tcl.gemm_fp8(a, s.double(), b, bs)),
        (ValueError, lambda: tcl.gemm_fp8(a, s[:, :1], b, bs)),
        (ValueError, lambda: tcl.gemm_fp8(a, s, b, torch.zeros(2, 2))),
        (ValueError, lambda: tcl.gemm_fp8(a, s, b[:, :128], bs)),
        (ValueError, lambda: tcl.gemm_fp8(a.t(), s, b, bs)),
        (TypeError, lambda: tcl.gemm_fp8(a, s, b, bs, out_dtype=torch.float16)),
        (ValueError, lambda: tcl.gemm_fp8(a[:, :0], s[:, :0], b[:, :0], bs[:, :0])),
        (ValueError, lambda: tcl.gemm_fp8_experts(a, s, w, ws, off)),                      # not on a GPU
        (ValueError, lambda: tcl.gemm_fp8_experts(a, s, w, ws, off[:2])),
        (TypeError, lambda: tcl.gemm_fp8_experts(a, s, w, ws, off.long())),
        (ValueError, lambda: tcl.gemm_fp8_experts(a, s, b, bs, off)),
        (ValueError, lambda: tcl.gemm_fp8_experts_wgrad(a, s, b, bs, off)),
        (ValueError, lambda: tcl.gemm_fp8_experts_wgrad(a, s, a[:, :128], s[:, :1], off)),
        (ValueError, lambda: tcl.gemm_fp8_experts_wgrad(a, s, a, s, off[:1])),
        (ValueError, lambda: tcl.quantize_fp8(x)),                                         # not on a GPU
        (ValueError, lambda: tcl.quantize_fp8(x, along="diagonal")),
        (ValueError, lambda: tcl.quantize_fp8(x, along="blocks", order=order)),
        (TypeError, lambda: tcl.quantize_fp8(x.half())),
        (ValueError, lambda: tcl.quantize_fp8(x[0])),
        (ValueError, lambda: tcl.quantize_fp8(x[:3], order=order)),
        (TypeError, lambda: tcl.sort_by_expert(ids.short(), 4)),
        (ValueError, lambda: tcl.sort_by_expert(ids, 0)),
        (ValueError, lambda: tcl.sort_by_expert(ids, 1025)),
        (ValueError, lambda: tcl.sort_by_expert(ids, 4, align=129)),
        (ValueError, lambda: tcl.sort_by_expert(ids.t(), 4)),
        (ValueError, lambda: tcl.sort_by_expert(ids, 4)),                                  # not on a GPU
        (ValueError, lambda: tcl.gather_rows(x[:2], order)),
        (ValueError, lambda: tcl.combine(x, None, order)),                                 # 4 rows, the order has 8
        (ValueError, lambda: tcl.combine(torch.zeros(8, 64), torch.zeros(4, 3), order)),
        (ValueError, lambda: tcl.combine_grad(x, torch.zeros(8, 64), None, order)),        # types differ
    ]:
        with pytest.raises(err):
            call()


def test_reference_e4m3_is_the_format():
    """The rounding used as the oracle against every e4m3 value and the midpoints between them."""
    bits = torch.arange(0, 127, dtype=torch.uint8)
    v = bits.view(torch.float8_e4m3fn).double().numpy()
    assert (ref.e4m3(v) == v).all() and (ref.e4m3(-v) == -v).all() and v[-1] == 448
    mid = (v[1:] + v[:-1]) / 2
    even = [v[i] if i % 2 == 0 else v[i + 1] for i in range(126)]
    assert (ref.e4m3(mid) == even).all()
    assert (ref.e4m3(mid * (1 + 1e-9)) == v[1:]).all() and (ref.e4m3(mid * (1 - 1e-9)) == v[:-1]).all()


def test_reference_order_by_hand():
    ids = torch.tensor([[1, 0], [2, -1], [1, 2]])
    assert ref.order(ids, 3, 2, 6 + 3) == ([0, 2, 4, 6], [2, 0, 4, -1, 3, 5], [1, -1, 0, 4, 2, 5, -1, -1, -1])
