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
and allocate their results on that stream.
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
X_BF16, X_F32 = 0, 1
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
    # (asking for the current stream's handle alone spares the wrapper object: 2 of a small call's microseconds)
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if device.index == torch.cuda.current_device():
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


def _device(name, first, *rest):
    """The GPU that ``first`` (called ``name``) is on; the others that are given have to be there too."""
    if not first.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device = first.device
    for t in rest:
        if t is not None and t.device != device:
            raise ValueError(f"all tensors must be on {device}, where {name} is, not on {t.device}")
    return device


def _x_type(t, name):
    if t.dtype == torch.bfloat16:
        return X_BF16
    if t.dtype == torch.float32:
        return X_F32
    raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def _ld(t, name, dim=2):
    """Leading dimension of a matrix (or of each of a batch) with contiguous rows."""
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    rows, cols = t.shape[-2:]
    if cols < 1:
        raise ValueError(f"{name} must have at least one column")
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous (stride(-1) == 1)")
    if rows > 1:
        if t.stride(-2) < cols:
            raise ValueError(f"{name}'s rows overlap")
        return t.stride(-2)
    return -(-cols // 16) * 16   # a single row never steps to a second one


def _int32(t, name, shape=None):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


def _order(order, tokens=None):
    offsets, position, source = order
    _int32(position, "position")
    _int32(source, "source")
    if position.dim() != 2 or source.dim() != 1:
        raise ValueError("position must be tokens x choices and source one row number per row")
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
    ldx = _ld(x, "x", 3 if batched and x.dim() == 3 else 2)
    rows, cols = x.shape[-2:]
    position = source = None
    top, made = 1, rows
    if order is not None:
        position, source = _order(order, rows)
        top, made = position.shape[1], source.shape[0]
    device = _device("x", x, position, source)
    pos, src = (position.data_ptr(), source.data_ptr()) if order is not None else (None, None)
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
    if data.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} must be float8_e4m3fn")
    if scale.dtype != torch.float32:
        raise TypeError(f"{name}'s scales must be float32")
    if scale.dim() != dim:
        raise ValueError(f"{name}'s scales must have {dim} dimensions")
    return _ld(data, name, dim)


def _kind(data, scale, name):
    """Whether scales belong to the rows of ``data`` or to blocks of 128 of them."""
    rows, cols = data.shape[-2:]
    groups = -(-cols // GROUP)
    if scale.shape[-1] != groups or scale.shape[:-2] != data.shape[:-2]:
        raise ValueError(f"{name} of shape {tuple(data.shape)} does not go with scales of shape {tuple(scale.shape)}")
    if scale.shape[-2] == rows:
        return SCALE_ROWS
    if scale.shape[-2] == -(-rows // GROUP):
        return SCALE_BLOCKS
    raise ValueError(f"{name} of shape {tuple(data.shape)} does not go with scales of shape {tuple(scale.shape)}")


def _out(dtype):
    if dtype is None or dtype == torch.bfloat16:
        return torch.bfloat16, OUT_BF16
    if dtype == torch.float32:
        return dtype, OUT_F32
    raise TypeError("the result is bfloat16 or float32")


def _result(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != shape or out.dtype != dtype:
        raise ValueError(f"out must be {dtype} of shape {shape}")
    return out


def gemm_fp8(a, a_scale, b, b_scale, out_dtype=None, out=None, stream=None):
    """C = A·Bᵀ (M x N; bf16 or ``out_dtype=torch.float32``) of e4m3 ``a`` (M x K, a scale for
    each row and 128 of K) and ``b`` (N x K, scales for its rows or for 128 x 128 blocks)."""
    lda, ldb = _operand(a, a_scale, "a"), _operand(b, b_scale, "b")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or N < 1:
        raise ValueError(f"shape mismatch: {tuple(a.shape)} and {tuple(b.shape)}")
    if tuple(a_scale.shape) != (M, -(-K // GROUP)):
        raise ValueError(f"a needs scales of shape {(M, -(-K // GROUP))}, not {tuple(a_scale.shape)}")
    kind = _kind(b, b_scale, "b")
    dtype, code = _out(out.dtype if out is not None else out_dtype)
    device = _device("a", a, a_scale, b, b_scale, out)
    with _on(stream):
        c = _result(out, (M, N), dtype, device)
        _call(_lib().gemm_fp8, "gemm_fp8", device, stream, M, N, K, a.data_ptr(), lda, a_scale.data_ptr(),
              a_scale.stride(0), a_scale.stride(1), b.data_ptr(), ldb, b_scale.data_ptr(), kind, b_scale.stride(0),
              b_scale.stride(1), c.data_ptr(), _ld(c, "out"), code)
    return c


def gemm_fp8_experts(a, a_scale, b, b_scale, offsets, out_dtype=None, out=None, stream=None):
    """C[r] = A[r]·B[e]ᵀ for the rows r of each expert e, ``offsets[e] <= r < offsets[e+1]``:
    ``a`` rows x K sorted by expert, ``b`` experts x N x K, ``offsets`` int32 on the GPU.
    Rows behind the last expert's are zeros. The gradient of ``a`` is the same product of the
    result's gradient with the transposed matrices (``quantize_fp8(w, along="blocks_t")``)."""
    lda, ldb = _operand(a, a_scale, "a"), _operand(b, b_scale, "b", 3)
    rows, K = a.shape
    experts, N = b.shape[:2]
    if b.shape[2] != K or N < 1 or experts < 1:
        raise ValueError(f"shape mismatch: {tuple(a.shape)} and {tuple(b.shape)}")
    if tuple(a_scale.shape) != (rows, -(-K // GROUP)):
        raise ValueError(f"a needs scales of shape {(rows, -(-K // GROUP))}, not {tuple(a_scale.shape)}")
    kind = _kind(b, b_scale, "b")
    _int32(offsets, "offsets", (experts + 1,))
    dtype, code = _out(out.dtype if out is not None else out_dtype)
    device = _device("a", a, a_scale, b, b_scale, offsets, out)
    with _on(stream):
        c = _result(out, (rows, N), dtype, device)
        _call(_lib().gemm_fp8_experts, "gemm_fp8_experts", device, stream, rows, experts, N, K, a.data_ptr(), lda,
              a_scale.data_ptr(), a_scale.stride(0), a_scale.stride(1), b.data_ptr(), ldb,
              b.stride(0) if experts > 1 else N * ldb, b_scale.data_ptr(), kind, b_scale.stride(0), b_scale.stride(1),
              b_scale.stride(2), offsets.data_ptr(), c.data_ptr(), _ld(c, "out"), code)
    return c


def gemm_fp8_experts_wgrad(a, a_scale, b, b_scale, offsets, out_dtype=None, out=None, stream=None):
    """C[e] = sum over expert e's rows r of A[:, r]·B[:, r]ᵀ (experts x N x K): the weights'
    gradients from ``a`` (N x rows) and ``b`` (K x rows), the result's gradient and the input
    quantised down the sorted rows (``quantize_fp8(..., along="columns")``). ``offsets`` are
    multiples of 128 (``sort_by_expert(..., align=128)``); experts without rows get zeros."""
    for t, s, name in ((a, a_scale, "a"), (b, b_scale, "b")):
        if t.dtype != torch.float8_e4m3fn:
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
    lda, ldb = (_ld(a, "a"), _ld(b, "b")) if rows else (0, 0)
    experts = offsets.numel() - 1
    if experts < 1:
        raise ValueError("offsets must have one entry more than there are experts")
    _int32(offsets, "offsets", (experts + 1,))
    dtype, code = _out(out.dtype if out is not None else out_dtype)
    device = _device("a", a, a_scale, b, b_scale, offsets, out)
    with _on(stream):
        c = _result(out, (experts, N, K), dtype, device)
        ldc = _ld(c, "out", 3)
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
    device = _device("ids", ids)
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
    xt, ldx = _x_type(x, "x"), _ld(x, "x")
    position, source = _order(order, x.shape[0])
    device = _device("x", x, position, source)
    with _on(stream):
        y = torch.empty((source.shape[0], x.shape[1]), dtype=x.dtype, device=device)
        _call(_lib().tcl_gather_rows, "gather_rows", device, stream, xt, x.shape[0], position.shape[1], y.shape[0],
              x.shape[1], x.data_ptr(), ldx, position.data_ptr(), source.data_ptr(), y.data_ptr(), x.shape[1])
    return y


def _weights(weights, position):
    if weights is None:
        return None
    if weights.dtype != torch.float32 or not weights.is_contiguous() or weights.shape != position.shape:
        raise ValueError(f"weights must be contiguous float32 of shape {tuple(position.shape)}")
    return weights.data_ptr()


def combine(y, weights, order: ExpertOrder, stream=None):
    """out[t] = sum over the token's slots j of weights[t, j]·y[position[t, j]] (None: ones), in
    fp32, rounded once to ``y``'s type. Dropped slots add nothing."""
    xt, ldy = _x_type(y, "y"), _ld(y, "y")
    position, source = _order(order)
    if y.shape[0] != source.shape[0]:
        raise ValueError(f"the order has {source.shape[0]} rows, y {y.shape[0]}")
    w = _weights(weights, position)
    device = _device("y", y, weights, position, source)
    tokens, top = position.shape
    with _on(stream):
        out = torch.empty((tokens, y.shape[1]), dtype=y.dtype, device=device)
        _call(_lib().tcl_combine, "combine", device, stream, xt, tokens, top, y.shape[0], y.shape[1], y.data_ptr(), ldy, w,
              position.data_ptr(), out.data_ptr(), y.shape[1])
    return out


def combine_grad(grad, y, weights, order: ExpertOrder, stream=None):
    """(gradient of ``y``, gradient of ``weights``) of ``combine`` from the gradient of its output:
    rows weights[t, j]·grad[t] (zeros in rows without a slot), and grad[t]·y[position[t, j]] in fp32."""
    xt, ldg, ldy = _x_type(grad, "grad"), _ld(grad, "grad"), _ld(y, "y")
    if y.dtype != grad.dtype or y.shape[1] != grad.shape[1]:
        raise ValueError("grad and y must have the same type and width")
    position, source = _order(order, grad.shape[0])
    if y.shape[0] != source.shape[0]:
        raise ValueError(f"the order has {source.shape[0]} rows, y {y.shape[0]}")
    w = _weights(weights, position)
    device = _device("grad", grad, y, weights, position, source)
    tokens, top = position.shape
    with _on(stream):
        dy = torch.empty((source.shape[0], y.shape[1]), dtype=y.dtype, device=device)
        dw = torch.empty((tokens, top), dtype=torch.float32, device=device)
        _call(_lib().tcl_combine_grad, "combine_grad", device, stream, xt, tokens, top, y.shape[0], y.shape[1],
              grad.data_ptr(), ldg, y.data_ptr(), ldy, w, position.data_ptr(), source.data_ptr(), dy.data_ptr(),
              y.shape[1], dw.data_ptr())
    return dy, dw
