"""Host side of the training operators and of the expert layer (no GPU needed)."""

import pytest
import torch

from fp8_block_scale_gb300.training import ExpertLayer


@pytest.fixture(scope="module")
def L():
    from fp8_block_scale_gb300 import _lib
    from fp8_block_scale_gb300.build import build
    build()
    _lib.load()
    return _lib


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_only_bf16_weights_are_quantised(L, dtype):
    """The kernel reads BF16 bits: another type would give wrong codes."""
    w = torch.zeros(2, 128, 128, dtype=dtype)
    q, s = torch.zeros(2, 128, 128, dtype=torch.uint8), torch.zeros(2, 1, 1)
    with pytest.raises(ValueError):
        L.moe_quantize_weight_128x128(w, q, s)
    layer = object.__new__(ExpertLayer)
    layer.models = [w, w]
    with pytest.raises(ValueError):
        layer.quantized()
