"""A language model's dense path on bf16 matrices, and its gradients: Python binding of
``include/tcl_dense.h``.

    out = gated_ffn(x, w_gate, w_up, w_down)                            # serving: prompts, single tokens
    out, kept = gated_ffn(x, w_gate, w_up, w_down, keep=True)           # training
    dx, dw_gate, dw_up, dw_down = gated_ffn_grad(grad, x, w_gate, w_up, w_down, kept)

    loss, lse = cross_entropy(x, w, targets)                            # logits x · wᵀ, never stored
    loss, lse, dx, dw = cross_entropy_grad(x, w, targets, grad)         # grad: each token's weight in the sum

    norm = clip_grads([dw_gate, dw_up, dw_down, dw], 1.0)               # in place

Weights are outputs × inputs, as a layer stores them. Matrices have contiguous rows, with any
distance between them; rows that start on 16-byte pieces are read in place, others are copied first.
Calls are asynchronous on ``stream`` (default: the current stream of the tensors' device) and
allocate their results and workspaces on that stream; nothing is kept between calls, so any of
them may be captured into a CUDA graph. Given another stream than the current one, the caller lets it
wait for whatever makes the operands (``stream.wait_stream``); the operands themselves may be
dropped right after the call.

The calls compute without a graph of autograd, also for tensors that require gradients: the
gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
import importlib.util
import warnings
from typing import NamedTuple

try:
    import torch
except ImportError:   # (the library itself needs no PyTorch; the calls below take its tensors)
    torch = None

from . import OUT_BF16, OUT_F32, TclError, _build, lib
from .fp8 import _INT, _device, _mat, _on, _too_large

__all__ = ["gated_ffn", "gated_ffn_grad", "GatedFfnKept", "cross_entropy", "cross_entropy_grad", "grad_norm", "clip_grads",
           "EXPORTED_SYMBOLS_DENSE"]

EXPORTED_SYMBOLS_DENSE = ("tcl_gated_ffn", "tcl_gated_ffn_grad", "tcl_cross_entropy", "tcl_cross_entropy_grad",
                          "tcl_grad_norm", "tcl_clip_gradients")
_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_CONFIG, _WORKSPACE = 8, 13   # TCL_ERR_CONFIG, TCL_ERR_WORKSPACE
if torch is not None:
    _BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    _TYPES = {_BF16: OUT_BF16, _F32: OUT_F32}   # (as tensors.cpp has them)

_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        I, P, F, Z = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
        L.tcl_gated_ffn.argtypes = [I, I, I, P, I, P, I, P, I, P, I, I, P, P, P, I, P, I, P, Z, P]
        L.tcl_gated_ffn_grad.argtypes = [I, I, I, P, I, P, I, P, I, P, I, P, I, I, P, P, P, I, P, I, P, I, P, I, P, I, I, P, Z, P]
        L.tcl_cross_entropy.argtypes = [I, I, I, P, I, P, I, P, I, P, P, P, Z, P]
        L.tcl_cross_entropy_grad.argtypes = [I, I, I, P, I, P, I, P, I, P, P, P, P, I, P, I, I, P, Z, P]
        L.tcl_grad_norm.argtypes = [I, P, P, P, P, P, Z, P]
        L.tcl_clip_gradients.argtypes = [I, P, P, P, P, F, P, P, Z, P]
        _bound = L
    return _bound


_native = None   # the binding's own module, once it is loaded; False where there is none


def _load():
    """The binding's own module for this Python and PyTorch, or False where there is none (a warning says why): the calls then
    go the way of those on a given stream, in some 15 us more of the host's time."""
    global _native
    if _native is not None:
        return _native
    L = _lib()
    path = _build.tensors_path()
    spec = importlib.util.spec_from_file_location(f"{__package__}._tensors", path)
    try:
        _tensors = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_tensors)
    except ImportError as e:
        warnings.warn(f"dense calls take more of the host's time without the binding's module: {e} (it is built by "
                      "`python -c 'import __graft_entry__ as g; g.build()'`)", RuntimeWarning, stacklevel=3)
        _native = False
        return _native
    _tensors.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                    for f in (L.tcl_gated_ffn, L.tcl_gated_ffn_grad, L.tcl_cross_entropy, L.tcl_cross_entropy_grad,
                              L.tcl_clip_gradients)))
    _native = _tensors
    return _native


class GatedFfnKept(NamedTuple):
    """What ``gated_ffn`` keeps for its gradients, bf16. (One buffer, of which views are made where they are asked
    for: four views cost as much of the host's time as the call's launches.)"""
    values: "torch.Tensor"   # 3 × tokens × a pitch of at least inner: hidden, gate, up  # noqa: F821
    inner: int

    @property
    def hidden(self):
        """act(gate) · up: tokens × inner."""
        return self.values[0, :, :self.inner]

    @property
    def gate(self):
        """x · w_gateᵀ: tokens × inner."""
        return self.values[1, :, :self.inner]

    @property
    def up(self):
        """x · w_upᵀ: tokens × inner."""
        return self.values[2, :, :self.inner]


def _call(fn, what, device, stream, room, *args):
    """Calls fn(*args, workspace, its size, stream) with a workspace of ``room`` bytes, and once more with a
    larger one where it asks for that."""
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(fn, what, device, stream, room, *args)
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    size = ctypes.c_size_t(room)
    space = torch.empty(room, dtype=torch.uint8, device=device) if room else None   # (on the stream: the caller is inside _on)
    st = fn(*args, space.data_ptr() if room else None, size, raw)
    if st == _WORKSPACE:
        space = torch.empty(size.value, dtype=torch.uint8, device=device)
        st = fn(*args, space.data_ptr(), size, raw)
    if st:
        raise TclError(st, what)


def _bf16(t, name):
    """(rows, columns, leading dimension) of a bf16 matrix."""
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    return _mat(t, name)


def _shape(rows, cols, want, name):
    if (rows, cols) != want:
        raise ValueError(f"{name} must be {want[0]} x {want[1]}, not {rows} x {cols}")


def _w_type(out_dtype):
    if out_dtype is None:
        out_dtype = _BF16
    code = _TYPES.get(out_dtype)
    if code is None:
        raise TypeError("weights' gradients are bfloat16 or float32")
    return out_dtype, code


def _ffn(x, w_gate, w_up, w_down, activation):
    """Checks of the block's operands: (tokens, hidden, inner, act), each one's leading dimension."""
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    tokens, hidden, ldx = _bf16(x, "x")
    inner, h, ldg = _bf16(w_gate, "w_gate")
    _shape(inner, h, (inner, hidden), "w_gate")
    r, h, ldu = _bf16(w_up, "w_up")
    _shape(r, h, (inner, hidden), "w_up")
    r, h, ldd = _bf16(w_down, "w_down")
    _shape(r, h, (hidden, inner), "w_down")
    if inner < 1:
        raise ValueError("the weights must have at least one row")
    return (tokens, hidden, inner, act), (ldx, ldg, ldu, ldd)


def gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu", keep: bool = False, stream=None):
    """out = (act(x · w_gateᵀ) * (x · w_upᵀ)) · w_downᵀ: tokens × hidden, bf16. ``w_gate`` and
    ``w_up`` are inner × hidden, ``w_down`` hidden × inner. ``activation``: "silu", "gelu" (with the
    normal distribution) or "gelu_tanh". The product in the middle is rounded to bf16.

    ``keep=True``: (out, kept) with what ``gated_ffn_grad`` needs."""
    if stream is None and (native := _native or _load()):
        done = native.gated_ffn(x, w_gate, w_up, w_down, _ACTIVATIONS.get(activation, -1), keep)
        if done is not None:   # (else: something to refuse, or another GPU than the current one)
            if done.__class__ is int:
                raise TclError(done, "gated_ffn")
            return (done[0], GatedFfnKept(done[1], w_gate.shape[0])) if keep else done
    (tokens, hidden, inner, act), (ldx, ldg, ldu, ldd) = _ffn(x, w_gate, w_up, w_down, activation)
    device = _device(stream, "x", x, w_gate, w_up, w_down)
    with _on(stream):
        pitch = (inner + 63) & ~63   # (rows on whole lines of 128 bytes)
        mid = torch.empty((3 if keep else 1, tokens, pitch), dtype=_BF16, device=device)
        out = torch.empty((tokens, hidden), dtype=_BF16, device=device)
        h = mid.data_ptr()
        part = 2 * tokens * pitch
        _call(_lib().tcl_gated_ffn, "gated_ffn", device, stream, 0, tokens, hidden, inner, x.data_ptr(), ldx, w_gate.data_ptr(),
              ldg, w_up.data_ptr(), ldu, w_down.data_ptr(), ldd, act, h + part if keep else None,
              h + 2 * part if keep else None, h, pitch, out.data_ptr(), hidden)
        return (out, GatedFfnKept(mid, inner)) if keep else out


def gated_ffn_grad(grad, x, w_gate, w_up, w_down, kept: GatedFfnKept, activation: str = "silu", out_dtype=None, stream=None):
    """(dx, dw_gate, dw_up, dw_down) of ``gated_ffn`` from the gradient of its result and what it
    kept. ``dx`` is bf16, the weights' gradients are bf16 or ``out_dtype=torch.float32``. The gradients
    of the two products in the middle are rounded to bf16."""
    if stream is None and (native := _native or _load()):
        done = native.gated_ffn_grad(grad, x, w_gate, w_up, w_down, *kept, _ACTIVATIONS.get(activation, -1),
                                     _TYPES.get(out_dtype or _BF16, -1))
        if done is not None:
            if done.__class__ is int:
                raise TclError(done, "gated_ffn_grad")
            return done
    (tokens, hidden, inner, act), (ldx, ldg, ldu, ldd) = _ffn(x, w_gate, w_up, w_down, activation)
    r, c, ld_grad = _bf16(grad, "grad")
    _shape(r, c, (tokens, hidden), "grad")
    dtype, code = _w_type(out_dtype)
    values, width = kept
    if values.dtype != _BF16:
        raise TypeError("kept.values must be bfloat16")
    shape = values.shape
    if len(shape) != 3 or shape[:2] != (3, tokens) or width != inner or shape[2] < inner or shape[2] % 8 or shape[2] > _INT or \
            not values.is_contiguous() or values.data_ptr() % 16:
        raise ValueError("kept must be as gated_ffn returned it for these operands")
    pitch = shape[2]
    device = _device(stream, "grad", grad, x, w_gate, w_up, w_down, values)
    with _on(stream):
        dx = torch.empty((tokens, hidden), dtype=_BF16, device=device)
        dw = [torch.empty(w.shape, dtype=dtype, device=device) for w in (w_gate, w_up, w_down)]
        h, part = values.data_ptr(), 2 * tokens * pitch
        room = 2 * ((2 * tokens * ((inner + 63) & ~63) + 255) & ~255)   # (what most sizes take: dgate and dup)
        _call(_lib().tcl_gated_ffn_grad, "gated_ffn_grad", device, stream, room, tokens, hidden, inner, grad.data_ptr(), ld_grad,
              x.data_ptr(), ldx, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, w_down.data_ptr(), ldd, act,
              h + part, h + 2 * part, h, pitch, dx.data_ptr(), hidden, dw[0].data_ptr(), hidden, dw[1].data_ptr(), hidden,
              dw[2].data_ptr(), inner, code)
    return dx, *dw


def _entropy(x, w, targets):
    tokens, hidden, ldx = _bf16(x, "x")
    vocab, h, ldw = _bf16(w, "w")
    _shape(vocab, h, (vocab, hidden), "w")
    if vocab < 1:
        raise ValueError("w must have at least one row")
    if targets.dtype not in (_I32, _I64):
        raise TypeError("targets must be int32 or int64")
    if tuple(targets.shape) != (tokens,) or not targets.is_contiguous():
        raise ValueError(f"targets must be contiguous of shape {(tokens,)}")
    return tokens, hidden, vocab, ldx, ldw


def cross_entropy(x, w, targets, stream=None):
    """(loss, lse) of the logits l = x · wᵀ (tokens × vocabulary), which are never stored: for each
    token lse = log Σ exp(l) and loss = lse - l[target], fp32. ``targets`` (int32 or int64) outside the
    vocabulary drop their token: its loss is 0. Logits beyond ±2^30 count as infinite."""
    if stream is None and (native := _native or _load()):
        done = native.cross_entropy(x, w, targets)
        if done is not None:
            if done.__class__ is int:
                raise TclError(done, "cross_entropy")
            return done
    tokens, hidden, vocab, ldx, ldw = _entropy(x, w, targets)
    device = _device(stream, "x", x, w, targets)
    with _on(stream):
        loss = torch.empty(tokens, dtype=_F32, device=device)
        lse = torch.empty(tokens, dtype=_F32, device=device)
        # (what operands on 16-byte pieces take: sums for each token and 64 words, for few tokens each warp of the GPU)
        room = tokens * (8 * max((vocab + 63) // 64, 1024 if tokens <= 128 else 0) + 4) + 512
        _call(_lib().tcl_cross_entropy, "cross_entropy", device, stream, room, tokens, hidden, vocab, x.data_ptr(), ldx, w.data_ptr(),
              ldw, targets.data_ptr(), targets.element_size(), loss.data_ptr(), lse.data_ptr())
    return loss, lse


def cross_entropy_grad(x, w, targets, grad, out_dtype=None, stream=None):
    """(loss, lse, dx, dw): ``cross_entropy`` and the gradients of Σ grad · loss, ``grad`` a float32
    weight for each token (1/tokens for a mean). Dropped tokens add nothing and get zeros. ``dx`` is
    bf16, ``dw`` bf16 or ``out_dtype=torch.float32``. The exponentials of the logits, computed once for
    both, are kept in bf16 for 2 GiB of them at a time."""
    if stream is None and (native := _native or _load()):
        done = native.cross_entropy_grad(x, w, targets, grad, _TYPES.get(out_dtype or _BF16, -1))
        if done is not None:
            if done.__class__ is int:
                raise TclError(done, "cross_entropy_grad")
            return done
    tokens, hidden, vocab, ldx, ldw = _entropy(x, w, targets)
    if grad.dtype != _F32:
        raise TypeError("grad must be float32")
    if tuple(grad.shape) != (tokens,) or not grad.is_contiguous():
        raise ValueError(f"grad must be contiguous of shape {(tokens,)}")
    dtype, code = _w_type(out_dtype)
    device = _device(stream, "x", x, w, targets, grad)
    with _on(stream):
        loss = torch.empty(tokens, dtype=_F32, device=device)
        lse = torch.empty(tokens, dtype=_F32, device=device)
        dx = torch.empty((tokens, hidden), dtype=_BF16, device=device)
        dw = torch.empty((vocab, hidden), dtype=dtype, device=device)
        # (what most sizes take: exponentials, scaled rows of x, sums for each 64 words and two more values a token)
        words = (vocab + 63) // 64
        room = tokens * (136 * words + 128 * ((hidden + 63) // 64) + 8) + 1280 if tokens * words <= 1 << 24 else 0
        _call(_lib().tcl_cross_entropy_grad, "cross_entropy_grad", device, stream, room, tokens, hidden, vocab, x.data_ptr(), ldx,
              w.data_ptr(), ldw, targets.data_ptr(), targets.element_size(), grad.data_ptr(), loss.data_ptr(), lse.data_ptr(),
              dx.data_ptr(), hidden, dw.data_ptr(), hidden, code)
    return loss, lse, dx, dw


def _look(tensors, name):
    """(addresses, lengths, types, GPU) of contiguous bf16 and fp32 tensors, the first three as bytes."""
    if len(tensors) > _INT:
        _too_large(name)
    if native := _native or _load():
        return native.look(tensors, name)
    for t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be tensors, not {type(t).__name__}")
        if t.dtype not in _TYPES:
            raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")
        if t.layout != torch.strided or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    n = len(tensors)
    gpus = {t.device.index if t.is_cuda else -1 for t in tensors}
    return (bytes((ctypes.c_uint64 * n)(*[t.data_ptr() for t in tensors])), bytes((ctypes.c_int64 * n)(*[t.numel() for t in tensors])),
            bytes((ctypes.c_int32 * n)(*[_TYPES[t.dtype] for t in tensors])), -1 if n == 0 else gpus.pop() if len(gpus) == 1 else -2)


def _where(stream, tensors, *gpus):
    """The GPU that all of them are on; they are recorded on ``stream`` as ``_device`` does."""
    if gpus[0] == -2 or gpus.count(gpus[0]) < len(gpus):
        raise ValueError("all tensors must be on one GPU")
    return _device(stream, "tensors", *(tensors if stream is not None else tensors[:1]))


_SHARED = "a result shares memory with another tensor"


def _clip_room(tensors):
    """A sum for each block of the launches that they take."""
    return 16384 * (len(tensors) // 256 + 2)


def grad_norm(tensors, stream=None):
    """The square root of the sum of all elements' squares over bf16 and fp32 tensors: an fp32 scalar
    on the GPU. The same tensors give the same bits."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("at least one tensor")
    *host, gpu = _look(tensors, "tensors")
    device = _where(stream, tensors, gpu)
    with _on(stream):
        norm = torch.empty((), dtype=_F32, device=device)
        _call(_lib().tcl_grad_norm, "grad_norm", device, stream, _clip_room(tensors), len(tensors), *host, norm.data_ptr())
    return norm


def clip_grads(tensors, max_norm: float, out=None, stream=None):
    """Scales the tensors, in place or into ``out`` (a list of tensors of the same lengths and types), by
    max_norm / norm where their ``grad_norm`` is larger than ``max_norm``; a norm that is infinite or
    NaN scales nothing. The factor is rounded to float32, its product with a value to float32 and then to the value's
    type. Returns the norm before, an fp32 scalar on the GPU. A result may be its own tensor, but
    shares no memory with another one."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("at least one tensor")
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    if out is not None:
        out = list(out)
    if stream is None and (native := _native or _load()):
        done = native.clip_grads(tensors, out, max_norm)
        if done is not None:
            if done.__class__ is not int:
                return done
            raise ValueError(_SHARED) if done == _CONFIG else TclError(done, "clip_grads")
    ptr, length, types, gpu = _look(tensors, "tensors")
    to, gpus, everything = ptr, (gpu,), tensors
    if out is not None:
        to, to_length, to_types, to_gpu = _look(out, "out")
        if to_length != length or to_types != types:
            raise ValueError("out must hold a tensor of the same length and type for each one")
        gpus, everything = (gpu, to_gpu), tensors + out
    device = _where(stream, everything, *gpus)
    with _on(stream):
        norm = torch.empty((), dtype=_F32, device=device)
        try:
            _call(_lib().tcl_clip_gradients, "clip_grads", device, stream, _clip_room(tensors), len(tensors), ptr, to, length, types,
                  max_norm, norm.data_ptr())
        except TclError as e:
            if e.status != _CONFIG:
                raise
            raise ValueError(_SHARED) from None
    return norm
