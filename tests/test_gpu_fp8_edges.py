"""Edges of the e4m3 quantising, products and routing on the GPU: padding beside non-finite values,
captures, threads, sizes past the grid's axes, pair tiles over several waves, operands off the
tensor copies' grid."""
from __future__ import annotations

import pytest
import torch

import fp8_reference as ref
import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


# ------------------------------------------------------------------------------ quantising

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("along", ["rows", "columns", "blocks", "blocks_t", "rows in order", "columns in order"])
def test_padding_is_zero_beside_non_finite_values(along, value, dtype):
    """The bytes between a row's end and the next multiple of 16 are zeros whatever the last group holds."""
    x = torch.randn(140, 203, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[139, 202] = value
    x[0, 202] = value
    x[139, 0] = value
    order = None
    if "order" in along:
        order = tcl.sort_by_expert(torch.zeros(140, 1, dtype=torch.int32, device=DEV), 1)
    data, scale = tcl.quantize_fp8(x.to(DEV), along=along.split()[0], order=order)
    rows, cols = data.shape
    pitch = -(-cols // 16) * 16
    assert pitch > cols and data.stride(0) == pitch
    padding = data.as_strided((rows, pitch), (pitch, 1)).view(torch.uint8)[:, cols:]
    assert bool((padding == 0).all())
    assert not bool(torch.isfinite(scale).all())      # (and the groups that hold the value carry it)
