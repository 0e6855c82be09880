"""The operators strung together as a training step uses them: gradients
against torch.autograd of the same layer in float64, a falling loss, and the
trained weights served in FP8."""

import os
import sys

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.training import ExpertLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("M,H,I,E,k,mask", [(7, 64, 24, 4, 2, False), (300, 200, 136, 9, 3, True), (64, 256, 128, 40, 8, False)])
def test_layer_gradients_match_autograd(M, H, I, E, k, mask):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    layer = ExpertLayer(M, H, I, E, k, generator=g)
    logits = torch.randn(M, E, device="cuda", generator=g)
    layer.route(logits)
    if mask:
        # mask some routes and plan again
        layer.topk_ids[::5, 1] = -1
        L.moe_plan(layer.topk_ids, E, layer.block_m, layer.sorted_ids, layer.expert_ids, layer.num_padded,
                   layer.plan_workspace)
        L.moe_plan_groups(layer.sorted_ids, layer.expert_ids, layer.num_padded, layer.block_m, M * k,
                          layer.group_start, layer.group_rows, layer.route_slot)
    x = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    dout = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    out = layer.forward(x).clone()
    dx, dwt = layer.backward(dout)

    xd = x.double().requires_grad_()
    w13, w2 = layer.w13.double().requires_grad_(), layer.w2.double().requires_grad_()
    wt = layer.topk_weights.double().requires_grad_()
    ids = layer.topk_ids.long()
    total = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gate, up = (xd[t] @ w13[e].t()).chunk(2, dim=1)
        h = torch.nn.functional.silu(gate) * up * wt[t, j][:, None]
        total = total.index_add(0, t, h @ w2[e].t())
    total.backward(dout.double())
    # every value passes at most five BF16 roundings on its way (u = 2^-8, of
    # random sign): a relative 2-norm of sqrt(5) * 2^-8 / sqrt(3) at most
    tol = 5 ** 0.5 / 256 / 3 ** 0.5 * 1.5
    assert _rel(out, total.detach()) < tol
    assert _rel(dx, xd.grad) < tol
    assert _rel(layer.grads[0], w13.grad) < tol and _rel(layer.grads[1], w2.grad) < tol
    live = ids >= 0
    assert _rel(dwt[live], wt.grad[live]) < tol
    assert (dwt[~live] == 0).all()
    assert int(layer.status.item()) == 0


def _reference_losses(steps, tokens, H, I, E, k, lr, seed):
    """The example's run in plain torch: FP32 weights, autograd and torch's AdamW."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    teacher = ExpertLayer(tokens, H, I, E, k, generator=gen)
    layer = ExpertLayer(tokens, H, I, E, k, generator=gen)
    w = [p.clone().requires_grad_() for p in layer.params]
    opt = torch.optim.AdamW(w, lr=lr, weight_decay=0.0)

    def run(w13, w2, x, ids, wt):
        y = torch.zeros(tokens, H, device="cuda")
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            gate, up = (x[t] @ w13[e].t()).chunk(2, dim=1)
            y = y.index_add(0, t, (torch.nn.functional.silu(gate) * up * wt[t, j][:, None]) @ w2[e].t())
        return y

    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, H, device="cuda", generator=gen).to(torch.bfloat16).float()
        logits = torch.randn(tokens, E, device="cuda", generator=gen)
        top, ids = logits.topk(k, dim=1)
        wt = torch.softmax(top, dim=1)
        want = run(*[p.detach() for p in teacher.params], x, ids, wt)
        loss = (run(*w, x, ids, wt) - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@pytest.mark.parametrize("bits", [32, 8])
def test_example_trains_like_plain_torch_and_serves(bits):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        from train_experts import train
    finally:
        sys.path.pop(0)
    size = dict(steps=40, tokens=512, H=256, I=128, E=8, top_k=2, lr=2e-3, seed=0)
    losses, trained, served = train(state_bits=bits, **size)
    size["k"] = size.pop("top_k")
    ref = _reference_losses(**size)
    assert losses[-1] < losses[0]
    # BF16 weights and activations put a relative error of about 1% on an output
    # whose error the loss squares; the gradients' noise of the same size moves
    # the path by less than that
    for a, b in zip(losses, ref):
        assert abs(a - b) < 0.03 * b
    # E4M3 weights and activations: a few percent
    assert _rel(served, trained.double()) < 0.1
