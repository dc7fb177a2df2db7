"""The example's mixture-of-experts layer: every call together, forward and backward."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    assert tcl.last_device_error() == (0, 0)


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=7, experts=5, top=3, hidden=130, inner=96),
                                   dict(tokens=1500, experts=4, top=2, hidden=512, inner=300)])
def test_layer_and_gradients_against_fp32(example, sizes):
    """e4m3 keeps 4 bits: a value is off by at most 2^-4 of itself, evenly spread by 2^-4/sqrt(3)/1.4
    or so, 0.026 in the root mean square. A result behind n rounded operands in a row is then off by
    about 0.026·sqrt(n) of its norm: n is 4 for the output (x, W_in, a, W_out), 5 for the router
    weights' gradients, and 7 at most for the others; twice that is allowed."""
    for name, d in example.distances(**sizes).items():
        assert d < 2 * 0.026 * 7 ** 0.5, (name, d)


def test_training_lowers_the_loss(example):
    torch.manual_seed(0)
    losses = example.train(steps=60)
    assert losses[-1] < 0.5 * losses[0], losses


def test_serving_and_training_layouts_agree(example):
    """The sorted layout's padding changes where rows lie, not what is computed for them."""
    layer = example.ExpertLayer(8, 256, 128)
    ids, weights = example.router(200, 8, 3, "cuda", 5)
    x = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    out = layer.forward(x, ids, weights)
    assert torch.equal(out, layer.forward(x, ids, weights, train=True)[0])


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=7, experts=5, top=3, hidden=130, inner=96),
                                   dict(tokens=1500, experts=4, top=2, hidden=512, inner=300)])
def test_each_result_within_its_own_roundings(example, sizes):
    """The distances of the test above, each held to the rounded operands behind it: 4 for the output (x,
    W_in, a, W_out), 5 for the router weights' gradients, 7 for the others."""
    for name, d in example.distances(**sizes).items():
        n = {"output": 4, "router weights": 5}.get(name, 7)
        assert d < 2 * 0.026 * n ** 0.5, (name, d)
