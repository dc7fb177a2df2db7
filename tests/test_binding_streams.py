"""The products' binding on the host: operands of a call on a given stream are recorded on it."""
from __future__ import annotations

from contextlib import nullcontext
from types import SimpleNamespace

import torch

import tensor_core_loop_gb300 as tcl


def test_operands_are_recorded_on_the_given_stream(monkeypatch):
    recorded = []
    fake = SimpleNamespace(**{name: lambda *args: 0 for name in ("gemm_bf16_ex", "gemm_tf32_ex", "gemm_s8_ex", "gemm_f32_simt")})
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.cuda, "device", lambda d: nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(tcl, "lib", lambda: fake)
    stream = SimpleNamespace(cuda_stream=1)
    for dtype, out in ((torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                       (torch.int8, torch.int32)):
        a, b, c = torch.zeros(4, 8, dtype=dtype), torch.zeros(8, 16, dtype=dtype), torch.zeros(4, 16, dtype=out)
        calls = [lambda st: tcl.gemm_into(a, b, c, stream=st)]
        if dtype == torch.float32:
            calls.append(lambda st: tcl.gemm_simt_into(a, b, c, stream=st))
        for call in calls:
            recorded.clear()
            call(stream)
            assert {p for p, _ in recorded} == {t.data_ptr() for t in (a, b, c)} and all(s is stream for _, s in recorded)
            recorded.clear()
            call(None)
            assert not recorded
        r = tcl.gemm(a, b, stream=stream)
        assert r.data_ptr() in {p for p, _ in recorded}
