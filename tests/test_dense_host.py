"""The dense path's entry points on the host (no GPU): exports, refusals of the C ABI before it touches a
device, the binding's checks, and the reference's gradients against differences."""
from __future__ import annotations

import ctypes
import os
import re
from contextlib import nullcontext

import pytest
import torch

import dense_reference as ref
import tensor_core_loop_gb300 as tcl
from tensor_core_loop_gb300 import dense

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, PO, P2, P4, P8 = (0x10000000 + i for i in (0, 1, 2, 4, 8))   # addresses of some alignments, never used
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from tensor_core_loop_gb300 import _build
    _build.build()
    return dense._lib()


def test_exports(L):
    text = open(os.path.join(ROOT, "include", "tcl_dense.h")).read()
    declared = set(re.findall(r"TCL_API\s+[\w\s\*]+?\b(\w+)\s*\(", text))
    assert declared == set(tcl.EXPORTED_SYMBOLS_DENSE)
    for name in declared:
        assert hasattr(L, name)
    assert f"TCL_ERR_WORKSPACE = {dense._WORKSPACE} " in open(os.path.join(ROOT, "include", "tcl_gemm.h")).read()
    assert tcl.STATUS[dense._WORKSPACE] == "TCL_ERR_WORKSPACE"
    assert L.tcl_status_string(dense._WORKSPACE).decode() != "unknown status"


def size(n=0):
    return ctypes.byref(ctypes.c_size_t(n))


BIG = 2 ** 31 - 1
MOST = 2 ** 31 - 2 ** 16


def ffn(L, **kw):
    d = dict(T=4, H=64, F=96, X=P, ldx=64, G=P, ldg=64, U=P, ldu=64, D=P, ldd=96, act=0, gate=P, up=P, h=P, ldk=96, out=P, ldo=64,
             ws=None, wsb=size())
    if kw.pop("names", None):
        return d
    d.update(kw)
    return L.tcl_gated_ffn(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=2 ** 30, F=2 ** 23, ldd=2 ** 23, ldk=2 ** 23), 2), (dict(T=2 ** 30, H=2 ** 23), 2),
    (dict(T=-1), 2), (dict(H=0), 2), (dict(F=0), 2), (dict(T=BIG), 2), (dict(F=BIG, ldd=BIG, ldk=BIG), 2), (dict(act=3), 8), (dict(act=-1), 8),
    (dict(X=None), 1), (dict(G=None), 1), (dict(U=None), 1), (dict(D=None), 1), (dict(h=None), 1), (dict(out=None), 1),
    (dict(gate=None), 1), (dict(up=None), 1), (dict(wsb=None), 1), (dict(wsb=size(256)), 1),
    (dict(ldx=63), 3), (dict(ldg=63), 3), (dict(ldu=63), 3), (dict(ldd=95), 3), (dict(ldo=63), 3), (dict(ldk=95), 3), (dict(ldk=100), 3),
    (dict(X=PO), 4), (dict(G=PO), 4), (dict(U=PO), 4), (dict(D=PO), 4), (dict(out=PO), 4), (dict(h=P8), 4), (dict(gate=P8), 4),
    (dict(up=P2), 4), (dict(ws=P8, wsb=size(4096)), 4)])
def test_ffn_refuses(L, kw, status):
    assert ffn(L, **kw) == status


@pytest.mark.parametrize("call,kw", [
    ("ffn", dict(H=2 ** 25 + 1)), ("ffn", dict(F=2 ** 25 + 1)), ("ffn_grad", dict(T=2 ** 25 + 1)), ("ffn_grad", dict(F=2 ** 26)),
    ("entropy", dict(H=2 ** 25 + 1)), ("entropy_grad", dict(H=2 ** 26)), ("entropy_grad", dict(V=2 ** 25 + 1))])
def test_sums_too_long_for_a_bounded_wait_are_refused(L, call, kw):
    far = dict.fromkeys([k for k in globals()[call](L, names=True) if k.startswith("ld")], 2 ** 27)
    assert globals()[call](L, **far, **kw) == 2
    assert globals()[call](L, **far, **{k: 2 ** 25 for k in kw}, **{"X": None}) == 1   # (as far as the next check)


def ffn_grad(L, **kw):
    d = dict(T=4, H=64, F=96, grad=P, ldgr=64, X=P, ldx=64, G=P, ldg=64, U=P, ldu=64, D=P, ldd=96, act=0, gate=P, up=P, h=P, ldk=96,
             dX=P, lddx=64, dG=P, lddg=64, dU=P, lddu=64, dD=P, lddd=96, wt=1, ws=None, wsb=size())
    if kw.pop("names", None):
        return d
    d.update(kw)
    return L.tcl_gated_ffn_grad(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 2), (dict(H=0), 2), (dict(F=0), 2), (dict(H=BIG), 2), (dict(act=7), 8), (dict(wt=2), 8),
    *[(dict([(k, None)]), 1) for k in ("grad", "X", "G", "U", "D", "gate", "up", "h", "dX", "dG", "dU", "dD", "wsb")],
    (dict(T=0, dG=None), 1), (dict(wsb=size(1)), 1),
    *[(dict([(k, 63)]), 3) for k in ("ldgr", "ldx", "ldg", "ldu", "lddx", "lddg", "lddu")],
    (dict(ldd=95), 3), (dict(lddd=95), 3), (dict(ldk=88), 3), (dict(ldk=97), 3),
    *[(dict([(k, PO)]), 4) for k in ("grad", "X", "G", "U", "D", "dX", "dG", "dU", "dD", "gate", "up", "h")],
    (dict(wt=0, dG=P2), 4), (dict(wt=0, dU=P2), 4), (dict(wt=0, dD=P2), 4), (dict(ws=P4, wsb=size(512)), 4)])
def test_ffn_grad_refuses(L, kw, status):
    assert ffn_grad(L, **kw) == status


def entropy(L, **kw):
    d = dict(T=4, H=64, V=100, X=P, ldx=64, W=P, ldw=64, y=P, yb=8, loss=P, lse=P, ws=None, wsb=size())
    if kw.pop("names", None):
        return d
    d.update(kw)
    return L.tcl_cross_entropy(*d.values(), None)


def entropy_grad(L, **kw):
    d = dict(T=4, H=64, V=100, X=P, ldx=64, W=P, ldw=64, y=P, yb=8, grad=P, loss=P, lse=P, dX=P, lddx=64, dW=P, lddw=64, wt=1, ws=None,
             wsb=size())
    if kw.pop("names", None):
        return d
    d.update(kw)
    return L.tcl_cross_entropy_grad(*d.values(), None)


@pytest.mark.parametrize("call", [entropy, entropy_grad])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 2), (dict(H=0), 2), (dict(V=0), 2), (dict(T=MOST), 2), (dict(V=BIG), 2), (dict(T=2 ** 29, V=2 ** 29), 2), (dict(yb=2), 8),
    *[(dict([(k, None)]), 1) for k in ("X", "W", "y", "loss", "lse", "wsb")], (dict(ldx=63), 3), (dict(ldw=63), 3),
    (dict(X=PO), 4), (dict(W=PO), 4), (dict(y=P4), 4), (dict(yb=4, y=P2), 4), (dict(loss=P2), 4), (dict(lse=P2), 4),
    (dict(ws=P8, wsb=size(512)), 4), (dict(wsb=size(512)), 1)])
def test_entropy_refuses(L, call, kw, status):
    assert call(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(grad=None), 1), (dict(dX=None), 1), (dict(dW=None), 1), (dict(T=0, dW=None), 1), (dict(lddx=63), 3), (dict(lddw=63), 3),
    (dict(grad=P2), 4), (dict(dX=PO), 4), (dict(dW=PO), 4), (dict(wt=0, dW=P2), 4), (dict(wt=5), 8)])
def test_entropy_grad_refuses(L, kw, status):
    assert entropy_grad(L, **kw) == status


def clip(L, ptrs=(P, P), to=(P, P), lengths=(4, 5), types=(0, 1), bound=1.0, norm=P, ws=None, wsb=0, count=None, norm_only=False):
    n = len(ptrs)
    a, b = (ctypes.c_void_p * n)(*ptrs), (ctypes.c_void_p * n)(*to)
    args = (n if count is None else count, a) + (() if norm_only else (b,)) + ((ctypes.c_longlong * n)(*lengths), (ctypes.c_int * n)(*types))
    args += () if norm_only else (bound,)
    return (L.tcl_grad_norm if norm_only else L.tcl_clip_gradients)(*args, norm, ws, size(wsb), None)


@pytest.mark.parametrize("norm_only", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 2), (dict(lengths=(4, -1)), 2), (dict(lengths=(4, 2 ** 50)), 2), (dict(types=(0, 2)), 8), (dict(ptrs=(P, None)), 1),
    (dict(ptrs=(P2, P)), 4), (dict(ptrs=(P, PO)), 4), (dict(norm=None), 1), (dict(norm=P2), 4), (dict(wsb=256), 1),
    (dict(ws=P8, wsb=256), 4)])
def test_clip_refuses(L, norm_only, kw, status):
    assert clip(L, norm_only=norm_only, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(bound=-1.0), 8), (dict(bound=float("nan")), 8), (dict(to=(None, P)), 1), (dict(to=(P2, P)), 4),
                                       (dict(to=(P, PO)), 4)])
def test_clip_refuses_its_own(L, kw, status):
    assert clip(L, **kw) == status


def test_binding_refuses():
    x, wg, wd = torch.zeros(4, 64, dtype=BF16), torch.zeros(96, 64, dtype=BF16), torch.zeros(64, 96, dtype=BF16)
    table, y, grad = torch.zeros(100, 64, dtype=BF16), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    kept = tcl.GatedFfnKept(torch.zeros(3, 4, 96, dtype=BF16), 96)
    for err, call in [
        (ValueError, lambda: tcl.gated_ffn(x, wg, wg, wd)),                                   # not on a GPU
        (ValueError, lambda: tcl.gated_ffn(x, wg, wg, wd, activation="relu")),
        (TypeError, lambda: tcl.gated_ffn(x.float(), wg, wg, wd)),
        (TypeError, lambda: tcl.gated_ffn(x, wg.half(), wg, wd)),
        (ValueError, lambda: tcl.gated_ffn(x[0], wg, wg, wd)),
        (ValueError, lambda: tcl.gated_ffn(x, wg, wg[:95], wd)),
        (ValueError, lambda: tcl.gated_ffn(x, wg[:, :63], wg, wd)),
        (ValueError, lambda: tcl.gated_ffn(x, wg, wg, wg)),
        (ValueError, lambda: tcl.gated_ffn(x, wd.t(), wg, wd)),                               # rows not contiguous
        (ValueError, lambda: tcl.gated_ffn(x, wg[:0], wg[:0], wd[:, :0])),
        (ValueError, lambda: tcl.gated_ffn(x[:, :0], wg[:, :0], wg[:, :0], wd[:0])),
        (ValueError, lambda: tcl.gated_ffn(x.expand(4, 64).as_strided((4, 64), (32, 1)), wg, wg, wd)),   # overlapping rows
        (ValueError, lambda: tcl.gated_ffn_grad(x, x, wg, wg, wd, kept)),                     # not on a GPU
        (ValueError, lambda: tcl.gated_ffn_grad(x[:3], x, wg, wg, wd, kept)),
        (TypeError, lambda: tcl.gated_ffn_grad(x.float(), x, wg, wg, wd, kept)),
        (TypeError, lambda: tcl.gated_ffn_grad(x, x, wg, wg, wd, kept, out_dtype=torch.float16)),
        (TypeError, lambda: tcl.gated_ffn_grad(x, x, wg, wg, wd, kept._replace(values=kept.values.float()))),
        *[(ValueError, lambda v=v: tcl.gated_ffn_grad(x, x, wg, wg, wd, kept._replace(**v))) for v in (
            dict(inner=95), dict(values=kept.values[:, :3]), dict(values=kept.values[:2]), dict(values=kept.values[..., :88]),
            dict(values=torch.zeros(3, 4, 100, dtype=BF16)), dict(values=torch.zeros(3, 4, 104, dtype=BF16)[..., :96]),
            dict(values=torch.zeros(3 * 4 * 96 + 8, dtype=BF16)[1:1153].view(3, 4, 96)))],
        (ValueError, lambda: tcl.cross_entropy(x, table, y)),                                 # not on a GPU
        (TypeError, lambda: tcl.cross_entropy(x, table.float(), y)),
        (TypeError, lambda: tcl.cross_entropy(x, table, y.short())),
        (ValueError, lambda: tcl.cross_entropy(x, table, y[:3])),
        (ValueError, lambda: tcl.cross_entropy(x, table, y[:, None])),
        (ValueError, lambda: tcl.cross_entropy(x, table[:, :32], y)),
        (ValueError, lambda: tcl.cross_entropy(x, table[:0], y)),
        (ValueError, lambda: tcl.cross_entropy(x, table, torch.zeros(8, dtype=torch.int64)[::2])),
        (ValueError, lambda: tcl.cross_entropy_grad(x, table, y, grad)),                      # not on a GPU
        (TypeError, lambda: tcl.cross_entropy_grad(x, table, y, grad.double())),
        (ValueError, lambda: tcl.cross_entropy_grad(x, table, y, grad[:3])),
        (ValueError, lambda: tcl.cross_entropy_grad(x, table, y, torch.zeros(8)[::2])),
        (TypeError, lambda: tcl.cross_entropy_grad(x, table, y, grad, out_dtype=torch.float64)),
        (ValueError, lambda: tcl.grad_norm([])),
        (ValueError, lambda: tcl.grad_norm([grad])),                                          # not on a GPU
        (TypeError, lambda: tcl.grad_norm([grad, grad.half()])),
        (ValueError, lambda: tcl.grad_norm([table.t()])),
        (ValueError, lambda: tcl.clip_grads([], 1.0)),
        (ValueError, lambda: tcl.clip_grads([grad], -1.0)),
        (ValueError, lambda: tcl.clip_grads([grad], float("nan"))),
        (ValueError, lambda: tcl.clip_grads([grad], 1.0)),                                    # not on a GPU
        (ValueError, lambda: tcl.clip_grads([grad, table, grad], 1.0)),                       # twice the same
        (ValueError, lambda: tcl.clip_grads([grad, grad[:0], grad + 1], 1.0, out=[grad, grad[:0], grad])),
        (ValueError, lambda: tcl.clip_grads([grad], 1.0, out=[])),
        (ValueError, lambda: tcl.clip_grads([grad], 1.0, out=[grad[:3]])),
        (ValueError, lambda: tcl.clip_grads([grad], 1.0, out=[x[0, :4]])),
    ]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("ptrs,to,lengths,types", [
    ((0, 4096), (8192, 8192), (4, 5), (0, 1)), ((0, 4096), (8192, 8204), (4, 5), (0, 1)), ((0, 16), (0, 14), (4, 5), (0, 1)),
    ((0, 4096), (4, 8192), (4, 5), (0, 1)), ((0, 4096), (4096, 0), (4, 4), (0, 0)), ((0, 4096), (8192, 10), (4, 5), (0, 1)),
    ((0, 64, 128), (0, 64, 78), (8, 8, 2), (0, 1, 1)), ((0, 64, 128), (256, 132, 512), (8, 8, 4), (0, 0, 1)),
    ((0, 0, 0), (64, 256, 15 * 4), (8, 8, 8), (0, 0, 0))])
def test_clip_refuses_results_in_other_tensors(L, ptrs, to, lengths, types):
    assert clip(L, ptrs=tuple(P + a for a in ptrs), to=tuple(P + a for a in to), lengths=lengths, types=types) == 8


@pytest.mark.parametrize("ptrs,to,lengths,types", [
    ((0, 16), (0, 16), (4, 5), (0, 1)), ((0, 16), (64, 80), (4, 5), (0, 1)), ((0, 0), (64, 128), (4, 4), (0, 0)),
    ((0, 0, 16), (0, 0, 16), (4, 0, 5), (0, 0, 1)), ((32, 0), (32, 48), (4, 4), (0, 0)),
    ((0, 64, 128), (0, 64, 80), (8, 8, 2), (0, 1, 1))])   # (the second one ends where the third one begins)
def test_clip_takes_results_beside_them(L, ptrs, to, lengths, types):
    """(As far as the device: there is none here, or too small a workspace.)"""
    if torch.cuda.is_available():
        pytest.skip("addresses that are none")
    assert clip(L, ptrs=tuple(P + a for a in ptrs), to=tuple(P + a for a in to), lengths=lengths, types=types) not in (0, 1, 2, 4, 8, 9)


def meta(shape, strides, dtype=BF16):
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused():
    far = 2 ** 31
    x, wg, wd = meta((2, 64), (64, 1)), meta((96, 64), (64, 1)), meta((64, 96), (96, 1))
    y, grad = meta((2,), (1,), torch.int64), meta((2,), (1,), F32)
    for call in (lambda: tcl.gated_ffn(meta((2, 64), (far, 1)), wg, wg, wd),
                 lambda: tcl.gated_ffn(meta((far, 64), (64, 1)), wg, wg, wd),
                 lambda: tcl.gated_ffn(x, meta((96, 64), (far, 1)), wg, wd),
                 lambda: tcl.cross_entropy(x, meta((far, 64), (64, 1)), y),
                 lambda: tcl.cross_entropy(meta((2, 64), (far, 1)), wg, y),
                 lambda: tcl.cross_entropy_grad(x, meta((96, 64), (far, 1)), y, grad)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_operands_are_recorded_on_the_given_stream(monkeypatch):
    """The caching allocator must know that the given stream reads them (it would hand their memory out
    again once the caller drops them)."""
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(dense, "_on", lambda stream: nullcontext())
    monkeypatch.setattr(dense, "_call", lambda *args: None)
    stream = object()
    x, wg, wu = torch.zeros(4, 64, dtype=BF16), torch.zeros(96, 64, dtype=BF16), torch.ones(96, 64, dtype=BF16)
    wd, gr = torch.zeros(64, 96, dtype=BF16), torch.zeros(4, 64, dtype=BF16)
    y, w = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    kept = tcl.GatedFfnKept(torch.zeros(3, 4, 96, dtype=BF16), 96)
    a, b, c, d = (torch.zeros(5) for _ in range(4))
    for call, tensors in (
        (lambda st: tcl.gated_ffn(x, wg, wu, wd, stream=st), [x, wg, wu, wd]),
        (lambda st: tcl.gated_ffn(x, wg, wu, wd, keep=True, stream=st), [x, wg, wu, wd]),
        (lambda st: tcl.gated_ffn_grad(gr, x, wg, wu, wd, kept, stream=st), [gr, x, wg, wu, wd, kept.values]),
        (lambda st: tcl.cross_entropy(x, wg, y, stream=st), [x, wg, y]),
        (lambda st: tcl.cross_entropy_grad(x, wg, y, w, stream=st), [x, wg, y, w]),
        (lambda st: tcl.grad_norm([a, b], stream=st), [a, b]),
        (lambda st: tcl.clip_grads([a, b], 1.0, stream=st), [a, b]),
        (lambda st: tcl.clip_grads([a, b], 1.0, out=[c, d], stream=st), [a, b, c, d]),
    ):
        recorded.clear()
        call(stream)
        assert {p for p, _ in recorded} >= {t.data_ptr() for t in tensors}
        assert all(st is stream for _, st in recorded)
        recorded.clear()
        call(None)
        assert not recorded


# ------------------------------------------------------------------------------ the reference itself

def differences(f, args, i, direction, h=1e-5):
    up, down = [list(args) for _ in range(2)]
    up[i] = args[i] + h * direction
    down[i] = args[i] - h * direction
    return (f(*up) - f(*down)) / (2 * h)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_reference_gradients_of_the_block_are_differences(act):
    g = torch.Generator().manual_seed(1)
    args = [torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 7), (6, 7), (6, 7), (7, 6))]
    grad = torch.randn(5, 7, generator=g, dtype=torch.float64)

    def f(x, wg, wu, wd):
        return ((ref.act_of(act, x @ wg.t())[0] * (x @ wu.t())) @ wd.t() * grad).sum()

    assert torch.equal(ref.gated_ffn(*args, act)[0].v, (ref.act_of(act, args[0] @ args[1].t())[0] * (args[0] @ args[2].t())) @ args[3].t())
    for i, d in enumerate(ref.gated_ffn_grad(grad, *args, act)):
        direction = torch.randn(*args[i].shape, generator=g, dtype=torch.float64)
        want = differences(f, args, i, direction)
        assert abs((d.v * direction).sum() - want) <= 1e-7 * (1 + abs(want))


def test_reference_gradients_of_the_entropy_are_differences():
    g = torch.Generator().manual_seed(2)
    args = [torch.randn(6, 5, generator=g, dtype=torch.float64), torch.randn(9, 5, generator=g, dtype=torch.float64)]
    y = torch.tensor([0, 8, 3, -100, 9, 4])
    grad = torch.rand(6, generator=g, dtype=torch.float64)

    def losses(x, w):
        l = x @ w.t()
        at = y.clamp(0, 8)
        return torch.where((y >= 0) & (y < 9), torch.logsumexp(l, 1) - l[torch.arange(6), at], 0.0)

    loss, lse, dx, dw = ref.cross_entropy(*args, y, grad)
    assert torch.allclose(loss.v, losses(*args), rtol=1e-14) and loss.v[3] == 0 and loss.v[4] == 0
    for i, d in enumerate((dx, dw)):
        direction = torch.randn(*args[i].shape, generator=g, dtype=torch.float64)
        want = differences(lambda *a: (losses(*a) * grad).sum(), args, i, direction)
        assert abs((d.v * direction).sum() - want) <= 1e-7 * (1 + abs(want))


def test_reference_finds_planted_mistakes():
    """The bounds are tight enough to tell a result that lacks a term from one that has it."""
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(*s, generator=g).to(BF16) for s in ((40, 64), (300, 64)))
    y = torch.randint(0, 300, (40,), generator=g)
    grad = torch.rand(40, generator=g) / 40
    loss, lse, dx, dw = ref.cross_entropy(x, w, y, grad)
    ref.within(dx.v.to(BF16), dx, "dx")
    l = x.double() @ w.double().t()
    p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True)) * grad[:, None].double()
    with pytest.raises(AssertionError):
        ref.within((p @ w.double()).to(BF16), dx, "without the target")
    with pytest.raises(AssertionError):
        ref.within((p[1:].t() @ x[1:].double()).to(BF16), dw, "without a token")
    x, wg, wu, wd = (torch.randn(*s, generator=g).to(BF16) for s in ((9, 64), (100, 64), (100, 64), (64, 100)))
    out = ref.gated_ffn(x, wg, wu, wd, "silu")[0]
    with pytest.raises(AssertionError):
        ref.within(ref.gated_ffn(x, wg[1:], wu[1:], wd[:, 1:], "silu")[0].v, out, "without a column")
