"""Host side of the layer's quantised weights (no GPU needed)."""

import pytest
import torch

from fp8_block_scale_gb300 import training
from fp8_block_scale_gb300.training import ExpertLayer


@pytest.fixture
def layer(monkeypatch):
    """A layer's weights alone; library calls fail the test."""
    class NoCalls:
        def __getattr__(self, name):
            pytest.fail(f"{name} was reached")

    monkeypatch.setattr(training, "L", NoCalls())
    layer = object.__new__(ExpertLayer)
    layer.models, layer._calls = [torch.zeros(2, 256, 128).bfloat16(), torch.zeros(2, 128, 128).bfloat16()], 0
    return layer


def test_quantised_weights_go_where_they_fit(layer):
    def good():
        return [torch.empty(2, 256, 128, dtype=torch.uint8), torch.empty(2, 2, 1), torch.empty(2, 128, 128, dtype=torch.uint8),
                torch.empty(2, 1, 1)]

    for i in range(4):
        for bad in (good()[i][:1], good()[i].half(), good()[i].reshape(-1)):
            out = good()
            out[i] = bad
            with pytest.raises(ValueError):
                layer.quantized(out=out)
    with pytest.raises(ValueError):
        layer.quantized(out=good()[:3])
    out = good()
    out[0] = torch.empty(2, 128, 256, dtype=torch.uint8).transpose(1, 2)
    with pytest.raises(ValueError):
        layer.quantized(out=out)


def test_versions_of_the_weights(layer):
    first = layer.weights_version()
    assert layer.weights_version() == first
    layer.models[1].add_(1)
    second = layer.weights_version()
    layer._calls += 1
    assert len({first, second, layer.weights_version()}) == 3
    with torch.inference_mode():
        layer.models[0] = torch.zeros(2, 256, 128).bfloat16()
    layer.weights_version()
