"""One expert layer over several steps: what a step leaves must not reach the next."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.training import ExpertLayer
from tests.test_gpu_train import BF16, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def _plan_again(layer):
    L.moe_plan(layer.topk_ids, layer.E, layer.block_m, layer.sorted_ids, layer.expert_ids, layer.num_padded,
               layer.plan_workspace)
    L.moe_plan_groups(layer.sorted_ids, layer.expert_ids, layer.num_padded, layer.block_m, layer.M * layer.top_k,
                      layer.group_start, layer.group_rows, layer.route_slot)


def test_a_route_masked_later_has_no_weight_gradient():
    g = gen(31)
    layer = ExpertLayer(40, 64, 24, 6, 3, generator=g)
    x = torch.randn(40, 64, device="cuda", generator=g).to(BF16)
    layer.route(torch.randn(40, 6, device="cuda", generator=g))
    layer.forward(x)
    _, dwt = layer.backward(x)
    assert (dwt != 0).all()
    layer.route(torch.randn(40, 6, device="cuda", generator=g))
    layer.topk_ids[::4, 1] = -1
    _plan_again(layer)
    layer.forward(x)
    _, dwt = layer.backward(x)
    live = layer.topk_ids >= 0
    assert (dwt[~live] == 0).all() and (dwt[live] != 0).all()
