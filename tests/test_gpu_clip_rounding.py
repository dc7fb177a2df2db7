"""Clipped values bit by bit, as the header says that they are rounded."""
from __future__ import annotations

import math

import pytest
import torch

import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bound", [0.1, 1.0, 3.7, 1e-3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,to", [(0, 0), (3, 3), (1, 2)])
def test_factor_and_product_are_rounded_to_fp32(dtype, bound, offset, to):
    """Whole numbers: their squares' sum is exact in fp32 and fp64, so that the norm is its root, rounded to fp64."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(71)
    ts = [torch.randint(-128, 129, (n + offset,), generator=g).to(dtype).cuda()[offset:] for n in (70001, 9, 4096)]
    out = [torch.zeros(t.numel() + to, dtype=dtype, device="cuda")[to:] for t in ts]
    norm = math.sqrt(sum(int((t.double() ** 2).sum()) for t in ts))
    bound = float(torch.tensor(bound, dtype=F32))
    f = torch.tensor(bound / norm, dtype=torch.float64).to(F32).cuda()
    assert float(tcl.clip_grads(ts, bound, out=out)) == float(torch.tensor(norm, dtype=F32))
    for t, o in zip(ts, out):
        assert torch.equal(o, (t.to(F32) * f).to(dtype))
    assert tcl.last_device_error() == (0, 0)
