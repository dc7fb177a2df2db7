"""e4m3 products with one fp32 scale for each 128 values, and the sorting of tokens by
expert around them: Python binding of ``include/tcl_fp8.h``.

    xq, xs = quantize_fp8(x)                                    # groups of 128 along the rows
    wq, ws = quantize_fp8(w, along="blocks")                    # 128 x 128, w: outputs x inputs
    y = gemm_fp8(xq, xs, wq, ws)                                # x · wᵀ, bf16

    order = sort_by_expert(ids, experts)                        # ids: tokens x choices
    xq, xs = quantize_fp8(x, order=order)                       # the tokens' rows, sorted
    y = gemm_fp8_experts(xq, xs, wq, ws, order.offsets)         # w: experts x outputs x inputs
    out = combine(y, weights, order)                            # tokens x outputs

An e4m3 matrix is a pair: its data (``torch.float8_e4m3fn``, rows contiguous) and its
scales (``torch.float32``, one column for each 128 columns of the data, any strides).
Calls are asynchronous on ``stream`` (default: the current stream of the tensors' device)
and allocate their results on that stream. Given another stream than the current one, the
caller lets it wait for whatever makes the operands (``stream.wait_stream``); the operands
themselves may be dropped right after the call. Operands off the 16-byte grid (base, leading
dimension, distance of experts' matrices) go through scratch of the library, which has to be in
place before a call is captured into a CUDA graph and which that graph's replays share; nothing
else here uses any.

The calls compute without a graph of autograd, also for tensors that require gradients: the
gradients are calls of their own (each docstring says which).
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import NamedTuple

try:
    import torch
except ImportError:   # (the library itself needs no PyTorch; the calls below take its tensors)
    torch = None

from . import OUT_BF16, OUT_F32, TclError, lib

__all__ = ["quantize_fp8", "gemm_fp8", "gemm_fp8_experts", "gemm_fp8_experts_wgrad", "sort_by_expert", "ExpertOrder",
           "gather_rows", "combine", "combine_grad", "EXPORTED_SYMBOLS_FP8", "MAX_EXPERTS"]

EXPORTED_SYMBOLS_FP8 = ("tcl_quantize_fp8_rows", "tcl_quantize_fp8_columns", "tcl_quantize_fp8_blocks", "gemm_fp8",
                        "gemm_fp8_experts", "gemm_fp8_experts_wgrad", "tcl_sort_by_expert", "tcl_gather_rows",
                        "tcl_combine", "tcl_combine_grad")
MAX_EXPERTS = 1024
GROUP = 128
if torch is not None:
    _F8, _F32, _BF16, _I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
    _X_TYPES = {_BF16: 0, _F32: 1}   # X_BF16, X_F32
    _OUT = {_BF16: OUT_BF16, _F32: OUT_F32}
SCALE_ROWS, SCALE_BLOCKS = 0, 1

_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        I, P, W = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong
        L.tcl_quantize_fp8_rows.argtypes = [I, I, I, P, I, P, I, P, I, P, I, P, W, W, P]
        L.tcl_quantize_fp8_columns.argtypes = [I, I, I, P, I, P, I, I, P, I, P, W, W, P]
        L.tcl_quantize_fp8_blocks.argtypes = [I, I, I, I, P, I, W, I, P, I, W, P, P]
        L.gemm_fp8.argtypes = [I, I, I, P, I, P, W, W, P, I, P, I, W, W, P, I, I, P]
        L.gemm_fp8_experts.argtypes = [I, I, I, I, P, I, P, W, W, P, I, W, P, I, W, W, W, P, P, I, I, P]
        L.gemm_fp8_experts_wgrad.argtypes = [I, I, I, I, P, I, P, W, W, P, I, P, W, W, P, P, I, W, I, P]
        L.tcl_sort_by_expert.argtypes = [I, I, P, I, I, I, I, P, P, P, P]
        L.tcl_gather_rows.argtypes = [I, I, I, I, I, P, I, P, P, P, I, P]
        L.tcl_combine.argtypes = [I, I, I, I, I, P, I, P, P, P, I, P]
        L.tcl_combine_grad.argtypes = [I, I, I, I, I, P, I, P, I, P, P, P, P, I, P, P]
        _bound = L
    return _bound


class ExpertOrder(NamedTuple):
    """Slots (a token's choice of an expert) sorted by expert; all int32 on the GPU."""
    offsets: "torch.Tensor"    # experts + 1: each expert's first row  # noqa: F821
    position: "torch.Tensor"   # tokens x choices: the slot's row, -1 for a dropped one  # noqa: F821
    source: "torch.Tensor"     # rows: the row's slot (token * choices + choice), -1 for a row without one  # noqa: F821


def _call(fn, what, device, stream, *args):
    # (asking for the current stream's handle alone spares its wrapper object: 2 of a small call's microseconds)
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        st = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            st = fn(*args, raw)
    if st:
        raise TclError(st, what)


_here = nullcontext()


def _on(stream):
    """Allocations inside belong to ``stream`` (None: the current one, nothing to do)."""
    return _here if stream is None else torch.cuda.stream(stream)


def _device(stream, name, first, *rest):
    """The GPU that ``first`` (called ``name``) is on; the others that are given have to be there too.
    All of them are recorded on ``stream`` (None: the current one, whose memory they may be): the
    caching allocator does not hand their memory out again while work on it may still use them."""
    if not first.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device = first.device
    for t in rest:
        if t is not None and t.device != device:
            raise ValueError(f"all tensors must be on {device}, where {name} is, not on {t.device}")
    if stream is not None:
        for t in (first, *rest):
            if t is not None:
                t.record_stream(stream)
    return device


def _x_type(t, name):
    code = _X_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")
    return code


_INT = 2 ** 31 - 1


def _too_large(name):
    """For numbers past _INT, of which ctypes would pass on the low 32 bits."""
    raise ValueError(f"{name}'s sizes and leading dimension must fit 32 bits")


def _mat(t, name, dim=2):
    """(rows, columns, leading dimension) of a matrix, or of each of a batch, with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    rows, cols = shape[-2], shape[-1]
    if cols < 1:
        raise ValueError(f"{name} must have at least one column")
    if cols > 1 and stride[-1] != 1:
        raise ValueError(f"{name}'s rows must be contiguous (stride(-1) == 1)")
    ld = stride[-2] if rows > 1 else (cols + 15) & ~15   # (a single row never steps to a second one)
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    if ld > _INT or rows > _INT or shape[0] > _INT:
        _too_large(name)
    return rows, cols, ld


def _int32(t, name, shape=None):
    if t.dtype != _I32:
        raise TypeError(f"{name} must be int32")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


def _order(order, tokens=None):
    _, position, source = order
    _int32(position, "position")
    _int32(source, "source")
    if position.dim() != 2 or source.dim() != 1:
        raise ValueError("position must be tokens x choices and source one row number per row")
    if position.shape[0] > _INT or position.shape[1] > _INT or source.shape[0] > _INT:
        _too_large("the order")
    if tokens is not None and position.shape[0] != tokens:
        raise ValueError(f"the order is of {position.shape[0]} tokens, not of {tokens}")
    return position, source


def _fp8(rows, cols, device, batch=None):
    """e4m3 rows at a pitch of whole 16-byte pieces, as the tensor copies of a product read them."""
    pitch = -(-cols // 16) * 16
    full = torch.empty((rows, pitch) if batch is None else (batch, rows, pitch), dtype=torch.float8_e4m3fn, device=device)
    return full if pitch == cols else full[..., :cols]


def quantize_fp8(x, along: str = "rows", order: ExpertOrder | None = None, stream=None):
    """(data, scale) of a bf16 or fp32 matrix ``x`` (rows x cols) in e4m3 with a scale
    s = max(max|x|/448, 2^-126) for each group of 128 values, data = e4m3(x·(1/s)).

    ``along="rows"``: groups along the rows; data rows x cols, scale rows x ceil(cols/128).
    ``along="columns"``: groups down the columns, stored transposed; data cols x rows, scale
    cols x ceil(rows/128): the operands of a weight gradient.
    ``along="blocks"``: a scale for each 128 x 128 block; ``x`` may be a batch of matrices.
    ``along="blocks_t"``: the same values and scales, stored transposed.

    ``order`` (rows and columns): the rows of the sorted layout instead, each token's row in
    the place of each of its slots, zeros in rows without a slot."""
    batched = along in ("blocks", "blocks_t")
    if along not in ("rows", "columns") and not batched:
        raise ValueError("along must be 'rows', 'columns', 'blocks' or 'blocks_t'")
    if order is not None and batched:
        raise ValueError("an order goes with rows or columns")
    xt = _x_type(x, "x")
    rows, cols, ldx = _mat(x, "x", 3 if batched and x.dim() == 3 else 2)
    position = source = pos = src = None
    top, made = 1, rows
    if order is not None:
        position, source = _order(order, rows)
        top, made = position.shape[1], source.shape[0]
        pos, src = position.data_ptr(), source.data_ptr()
    device = _device(stream, "x", x, position, source)
    with _on(stream):
        if along == "rows":
            data = _fp8(made, cols, device)
            scale = torch.empty_strided((made, -(-cols // GROUP)), (1, made), dtype=torch.float32, device=device)
            _call(_lib().tcl_quantize_fp8_rows, "quantize_fp8", device, stream, xt, rows, cols, x.data_ptr(), ldx, pos, top,
                  src, made, data.data_ptr(), -(-cols // 16) * 16, scale.data_ptr(), 1, made)
            return data, scale
        if along == "columns":
            data = _fp8(cols, made, device) if made else torch.empty((cols, 0), dtype=torch.float8_e4m3fn, device=device)
            scale = torch.empty_strided((cols, -(-made // GROUP)), (1, cols), dtype=torch.float32, device=device)
            _call(_lib().tcl_quantize_fp8_columns, "quantize_fp8", device, stream, xt, rows, cols, x.data_ptr(), ldx, src,
                  top, made, data.data_ptr(), -(-made // 16) * 16, scale.data_ptr(), 1, cols)
            return data, scale
        turned = along == "blocks_t"
        batch = x.shape[0] if x.dim() == 3 else None
        qr, qc = (cols, rows) if turned else (rows, cols)
        data = _fp8(qr, qc, device, batch)
        blocks = (-(-qr // GROUP), -(-qc // GROUP))
        scale = torch.empty(blocks if batch is None else (batch,) + blocks, dtype=torch.float32, device=device)
        pitch = -(-qc // 16) * 16
        _call(_lib().tcl_quantize_fp8_blocks, "quantize_fp8", device, stream, xt, 1 if batch is None else batch, rows, cols,
              x.data_ptr(), ldx, 0 if batch is None else x.stride(0), int(turned), data.data_ptr(), pitch, qr * pitch,
              scale.data_ptr())
        return data, scale


def _operand(data, scale, name, dim=2):
    """(rows, columns, leading dimension, the scales' shape) of an e4m3 matrix."""
    if data.dtype != _F8:
        raise TypeError(f"{name} must be float8_e4m3fn")
    if scale.dtype != _F32:
        raise TypeError(f"{name}'s scales must be float32")
    shape = scale.shape
    if len(shape) != dim:
        raise ValueError(f"{name}'s scales must have {dim} dimensions")
    return *_mat(data, name, dim), shape


def _kind(rows, cols, shape, name):
    """Whether scales of this shape belong to rows of a matrix or to blocks of 128 of them."""
    if shape[-1] == -(-cols // GROUP):
        if shape[-2] == rows:
            return SCALE_ROWS
        if shape[-2] == -(-rows // GROUP):
            return SCALE_BLOCKS
    raise ValueError(f"{name} of {rows} x {cols} does not go with scales of shape {tuple(shape)}")


def _out_type(out, out_dtype, shape):
    """(type, its code) of a result: ``out``'s, or ``out_dtype`` (None: bf16)."""
    if out is not None:
        if tuple(out.shape) != shape or out_dtype not in (None, out.dtype):
            raise ValueError(f"out must be {out_dtype or out.dtype} of shape {shape}")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = _BF16
    code = _OUT.get(out_dtype)
    if code is None:
        raise TypeError("the result is bfloat16 or float32")
    return out_dtype, code


def gemm_fp8(a, a_scale, b, b_scale, out_dtype=None, out=None, stream=None):
    """C = A·Bᵀ (M x N; bf16 or ``out_dtype=torch.float32``) of e4m3 ``a`` (M x K, a scale for
    each row and 128 of K) and ``b`` (N x K, scales for its rows or for 128 x 128 blocks). Gradients are
    products of the same form: of ``a`` with ``b`` transposed (``quantize_fp8(b, along="blocks_t")``), of
    ``b`` with both operands quantised down the rows (``along="columns"``)."""
    M, K, lda, sa = _operand(a, a_scale, "a")
    N, k, ldb, sb = _operand(b, b_scale, "b")
    if k != K or N < 1:
        raise ValueError(f"shape mismatch: {tuple(a.shape)} and {tuple(b.shape)}")
    if sa[0] != M or sa[1] != -(-K // GROUP):
        raise ValueError(f"a needs scales of shape {(M, -(-K // GROUP))}, not {tuple(sa)}")
    kind = _kind(N, K, sb, "b")
    dtype, code = _out_type(out, out_dtype, (M, N))
    ldc = N if out is None else _mat(out, "out")[2]
    device = _device(stream, "a", a, a_scale, b, b_scale, out)
    with _on(stream):
        c = torch.empty((M, N), dtype=dtype, device=device) if out is None else out
        _call(_lib().gemm_fp8, "gemm_fp8", device, stream, M, N, K, a.data_ptr(), lda, a_scale.data_ptr(),
              *a_scale.stride(), b.data_ptr(), ldb, b_scale.data_ptr(), kind, *b_scale.stride(), c.data_ptr(), ldc, code)
    return c


def gemm_fp8_experts(a, a_scale, b, b_scale, offsets, out_dtype=None, out=None, stream=None):
    """C[r] = A[r]·B[e]ᵀ for the rows r of each expert e, ``offsets[e] <= r < offsets[e+1]``:
    ``a`` rows x K sorted by expert, ``b`` experts x N x K, ``offsets`` int32 on the GPU.
    Rows behind the last expert's are zeros. Offsets that do not ascend from 0 within the rows write
    nothing and are reported by ``last_device_error``. The gradient of ``a`` is the same product of the
    result's gradient with the transposed matrices (``quantize_fp8(w, along="blocks_t")``)."""
    rows, K, lda, sa = _operand(a, a_scale, "a")
    N, k, ldb, sb = _operand(b, b_scale, "b", 3)
    experts = b.shape[0]
    if k != K or N < 1 or experts < 1:
        raise ValueError(f"shape mismatch: {tuple(a.shape)} and {tuple(b.shape)}")
    if sa[0] != rows or sa[1] != -(-K // GROUP):
        raise ValueError(f"a needs scales of shape {(rows, -(-K // GROUP))}, not {tuple(sa)}")
    if sb[0] != experts:
        raise ValueError(f"b of {experts} experts does not go with scales of shape {tuple(sb)}")
    kind = _kind(N, K, sb, "b")
    _int32(offsets, "offsets", (experts + 1,))
    dtype, code = _out_type(out, out_dtype, (rows, N))
    ldc = N if out is None else _mat(out, "out")[2]
    device = _device(stream, "a", a, a_scale, b, b_scale, offsets, out)
    with _on(stream):
        c = torch.empty((rows, N), dtype=dtype, device=device) if out is None else out
        _call(_lib().gemm_fp8_experts, "gemm_fp8_experts", device, stream, rows, experts, N, K, a.data_ptr(), lda,
              a_scale.data_ptr(), *a_scale.stride(), b.data_ptr(), ldb, b.stride(0) if experts > 1 else N * ldb,
              b_scale.data_ptr(), kind, *b_scale.stride(), offsets.data_ptr(), c.data_ptr(), ldc, code)
    return c


def gemm_fp8_experts_wgrad(a, a_scale, b, b_scale, offsets, out_dtype=None, out=None, stream=None):
    """C[e] = sum over expert e's rows r of A[:, r]·B[:, r]ᵀ (experts x N x K): the weights'
    gradients from ``a`` (N x rows) and ``b`` (K x rows), the result's gradient and the input
    quantised down the sorted rows (``quantize_fp8(..., along="columns")``). ``offsets`` are
    multiples of 128 (``sort_by_expert(..., align=128)``), reported as above where they are not;
    experts without rows get zeros."""
    for t, s, name in ((a, a_scale, "a"), (b, b_scale, "b")):
        if t.dtype != _F8:
            raise TypeError(f"{name} must be float8_e4m3fn")
        if t.dim() != 2 or s.dim() != 2:
            raise ValueError(f"{name} and its scales must have 2 dimensions")
        if s.dtype != torch.float32:
            raise TypeError(f"{name}'s scales must be float32")
        if tuple(s.shape) != (t.shape[0], -(-t.shape[1] // GROUP)):
            raise ValueError(f"{name} of shape {tuple(t.shape)} does not go with scales of shape {tuple(s.shape)}")
    N, rows = a.shape
    K = b.shape[0]
    if b.shape[1] != rows or N < 1 or K < 1:
        raise ValueError(f"shape mismatch: {tuple(a.shape)} and {tuple(b.shape)}")
    lda, ldb = (_mat(a, "a")[2], _mat(b, "b")[2]) if rows else (0, 0)
    experts = offsets.numel() - 1
    if experts < 1:
        raise ValueError("offsets must have one entry more than there are experts")
    _int32(offsets, "offsets", (experts + 1,))
    dtype, code = _out_type(out, out_dtype, (experts, N, K))
    ldc = _mat(out, "out", 3)[2] if out is not None else K if N > 1 else (K + 15) & ~15
    device = _device(stream, "a", a, a_scale, b, b_scale, offsets, out)
    with _on(stream):
        c = torch.empty((experts, N, K), dtype=dtype, device=device) if out is None else out
        _call(_lib().gemm_fp8_experts_wgrad, "gemm_fp8_experts_wgrad", device, stream, rows, experts, N, K, a.data_ptr(),
              lda, a_scale.data_ptr(), a_scale.stride(0), a_scale.stride(1), b.data_ptr(), ldb, b_scale.data_ptr(),
              b_scale.stride(0), b_scale.stride(1), offsets.data_ptr(), c.data_ptr(), ldc,
              c.stride(0) if experts > 1 else N * ldc, code)
    return c


def sort_by_expert(ids, experts: int, align: int = 1, stream=None) -> ExpertOrder:
    """The order of the slots of ``ids`` (tokens x choices, int32 or int64; anything outside
    0 .. experts-1 drops the slot) by expert, and by slot within an expert. Each expert's rows
    are padded to a multiple of ``align``: 1 for a forward pass, 128 where weight gradients are
    to follow."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64")
    if ids.dim() != 2 or ids.shape[1] < 1 or not ids.is_contiguous():
        raise ValueError("ids must be tokens x choices, contiguous")
    if not 1 <= experts <= MAX_EXPERTS or not 1 <= align <= 128:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, an align of 1 to 128")
    tokens, top = ids.shape
    slots = tokens * top
    rows = (slots + min(experts, slots) * (align - 1)) // align * align
    if tokens > _INT or top > _INT or rows > _INT:
        _too_large("the order")
    device = _device(stream, "ids", ids)
    with _on(stream):
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=device)
        position = torch.empty((tokens, top), dtype=torch.int32, device=device)
        source = torch.empty(rows, dtype=torch.int32, device=device)
        _call(_lib().tcl_sort_by_expert, "sort_by_expert", device, stream, tokens, top, ids.data_ptr(), ids.element_size(),
              experts, align, rows, offsets.data_ptr(), position.data_ptr(), source.data_ptr())
    return ExpertOrder(offsets, position, source)


def gather_rows(x, order: ExpertOrder, stream=None):
    """The tokens' rows of ``x`` (bf16 or fp32) in sorted order, zeros in rows without a slot.
    Its gradient is ``combine(d_rows, None, order)``."""
    xt = _x_type(x, "x")
    tokens, cols, ldx = _mat(x, "x")
    position, source = _order(order, tokens)
    rows = source.shape[0]
    device = _device(stream, "x", x, position, source)
    with _on(stream):
        y = torch.empty((rows, cols), dtype=x.dtype, device=device)
        _call(_lib().tcl_gather_rows, "gather_rows", device, stream, xt, tokens, position.shape[1], rows, cols,
              x.data_ptr(), ldx, position.data_ptr(), source.data_ptr(), y.data_ptr(), cols)
    return y


def _weights(weights, position):
    if weights is None:
        return None
    if weights.dtype != _F32 or not weights.is_contiguous() or weights.shape != position.shape:
        raise ValueError(f"weights must be contiguous float32 of shape {tuple(position.shape)}")
    return weights.data_ptr()


def combine(y, weights, order: ExpertOrder, stream=None):
    """out[t] = sum over the token's slots j of weights[t, j]·y[position[t, j]] (None: ones), in
    fp32, rounded once to ``y``'s type. Dropped slots add nothing. Gradients: ``combine_grad``."""
    xt = _x_type(y, "y")
    rows, cols, ldy = _mat(y, "y")
    position, source = _order(order)
    if rows != source.shape[0]:
        raise ValueError(f"the order has {source.shape[0]} rows, y {rows}")
    w = _weights(weights, position)
    device = _device(stream, "y", y, weights, position, source)
    tokens, top = position.shape
    with _on(stream):
        out = torch.empty((tokens, cols), dtype=y.dtype, device=device)
        _call(_lib().tcl_combine, "combine", device, stream, xt, tokens, top, rows, cols, y.data_ptr(), ldy, w,
              position.data_ptr(), out.data_ptr(), cols)
    return out


def combine_grad(grad, y, weights, order: ExpertOrder, stream=None):
    """(gradient of ``y``, gradient of ``weights``) of ``combine`` from the gradient of its output:
    rows weights[t, j]·grad[t] (zeros in rows without a slot), and grad[t]·y[position[t, j]] in fp32."""
    xt, ldg = _x_type(grad, "grad"), _mat(grad, "grad")[2]
    rows, cols, ldy = _mat(y, "y")
    if y.dtype != grad.dtype or y.shape[1] != grad.shape[1]:
        raise ValueError("grad and y must have the same type and width")
    position, source = _order(order, grad.shape[0])
    if rows != source.shape[0]:
        raise ValueError(f"the order has {source.shape[0]} rows, y {rows}")
    w = _weights(weights, position)
    device = _device(stream, "grad", grad, y, weights, position, source)
    tokens, top = position.shape
    with _on(stream):
        dy = torch.empty((rows, cols), dtype=y.dtype, device=device)
        dw = torch.empty((tokens, top), dtype=torch.float32, device=device)
        _call(_lib().tcl_combine_grad, "combine_grad", device, stream, xt, tokens, top, rows, cols, grad.data_ptr(), ldg,
              y.data_ptr(), ldy, w, position.data_ptr(), source.data_ptr(), dy.data_ptr(), cols, dw.data_ptr())
    return dy, dw
