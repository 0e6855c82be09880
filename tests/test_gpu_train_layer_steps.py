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


def test_a_skipped_step_does_not_count():
    """A skipped first step, then one from new gradients, is the same as that step alone."""
    layers = [ExpertLayer(8, 64, 24, 3, 2, weight_decay=0.1, generator=gen(5)) for _ in range(2)]
    flag = torch.ones(1, dtype=torch.int32, device="cuda")
    for grad in layers[0].grads:
        grad.copy_(torch.randn(grad.shape, device="cuda", generator=gen(6)))
    layers[0].step(1e-2, skip=flag)
    layers[0].step(1e-2, skip=flag)
    for a, b in zip(layers[0].params, layers[1].params):
        assert torch.equal(a, b)
    for k in range(3):
        for layer in layers:
            for i, grad in enumerate(layer.grads):
                grad.copy_(torch.randn(grad.shape, device="cuda", generator=gen(7 + 10 * k + i)))
        flag.zero_()
        layers[0].step(1e-2, skip=flag if k == 0 else None)
        layers[1].step(1e-2)
        for a, b in zip(layers[0].params + layers[0].models, layers[1].params + layers[1].models):
            assert torch.equal(a, b), k
    assert layers[0].steps == layers[1].steps == 3


def test_backward_needs_its_forward():
    """The gradient of pre takes pre's place: a second backward would run on gradients."""
    layer = ExpertLayer(8, 64, 24, 3, 2, generator=gen(8))
    x = torch.randn(8, 64, device="cuda", generator=gen(9)).to(BF16)
    logits = torch.randn(8, 3, device="cuda", generator=gen(10))
    layer.route(logits)
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    layer.backward(x)
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    layer.route(logits)
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    layer.forward(x)
    layer.backward(x)
