"""Routing by scores and the norms through the bounds-checking build: results as in the normal
build, and no check fails."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.build import build
from tests import test_gpu_block_norm as N
from tests import test_gpu_block_route as R

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


@pytest.mark.parametrize("case", [R.CASES[i] for i in (0, 1, 5, 8, 11)])
def test_routes(case):
    R.test_choice_and_weights(*case)


def test_route_edges():
    R.test_values_near_or_equal("few values")
    R.test_left_out_experts_empty_rows_and_padding()
    R.test_gradient_of_repeated_unlisted_and_left_out_experts()


@pytest.mark.parametrize("M,H", [(3, 8), (17, 256), (7, 1160), (5, 8200)])
def test_norms(M, H):
    N.test_forward_widths(M, H)
    N.test_backward_widths(M, H)
