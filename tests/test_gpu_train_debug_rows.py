"""The row kernels and AdamW through the bounds-checking build: results as in
the normal build, and no check fails."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.build import build
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


def test_plan_groups():
    T.test_groups_of_a_plan_match_the_reference()


@pytest.mark.parametrize("M,k,width", [(1, 1, 8), (300, 9, 264)])
def test_gather_and_sum(M, k, width):
    T.test_gather_and_sum(M, k, width, T.BF16)
    T.test_gather_without_tokens_and_sum_without_rows()


@pytest.mark.parametrize("kind", ["routes", "slots", "in place"])
def test_swiglu_backward(kind):
    T.test_swiglu_backward(77, 256, T.FP16, kind)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    T.test_adamw_step(bits, T.BF16, T.BF16)
    T.test_adamw_with_gradients_of_several_types()


@pytest.mark.parametrize("slots,K,N", [(9, 5000, 320), (1, 7168, 512)])
def test_few_slots(slots, K, N):
    T.test_few_slots_with_long_and_short_contractions(slots, K, N)


def test_counts_stay_at_zero_on_an_arguments_mismatch():
    """More chunks than the table has are left out before any access."""
    for bits in (32, 8):
        ts = T._tensors([3000], bits, T.F32, T.BF16, T.gen(1))
        args = L.make_adamw_args(L.AdamWTable(ts), seed=1, **T.HYPER)
        args.chunks += 1000
        L.moe_adamw_step(args)
        torch.cuda.synchronize()
