"""The training side through the bounds-checking build: results as in the
normal build, and no check fails."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.build import build
from fp8_block_scale_gb300.training import ExpertLayer
from tests import test_gpu_train as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _debug_library():
    build(debug_bounds=True)
    with L.use_library(L.LIB_DEBUG_PATH):
        assert L.moe_debug_bounds_enabled()
        L.moe_debug_bounds_read(reset=True)
        yield


@pytest.fixture(autouse=True)
def _no_failures():
    yield
    n, f, line = L.moe_debug_bounds_read(reset=True)
    assert n == 0, f"{n} bounds checks failed, first at {f}:{line}"


@pytest.mark.parametrize("counts,K,N", [T.SHAPES[i] for i in (1, 2, 5, 6, 9)])
def test_grouped_products(counts, K, N):
    T.test_grouped_forward_and_input_gradient(counts, K, N, T.BF16)
    T.test_grouped_swiglu_epilogue(counts, K, N, T.FP16, "routes")
    T.test_grouped_wgrad(counts, K, N, T.BF16, T.F32)


def test_bad_groups():
    T.test_bad_groups_are_reported_and_skipped()


def test_layer_step():
    layer = ExpertLayer(100, 128, 72, 12, 3, state_bits=8)
    layer.route(torch.randn(100, 12, device="cuda"))
    x = torch.randn(100, 128, device="cuda").to(torch.bfloat16)
    layer.forward(x)
    layer.backward(x)
    layer.step(1e-3)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
