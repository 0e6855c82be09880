"""A block's passes under torch.autocast: its own types, as without."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from tests.test_gpu_block_layer import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_autocast_changes_nothing(dtype):
    results = []
    for enabled in (False, True):
        b, x, dout = make(48, 256, 128, 8, 2, 51)
        with torch.autocast("cuda", dtype=dtype, enabled=enabled):
            out = b.forward(x).clone()
            dx = b.backward(dout).clone()
        results.append([out, dx, *b.grads.values(), *b.layer.grads])
    assert all(torch.equal(a, w) for a, w in zip(*results))
