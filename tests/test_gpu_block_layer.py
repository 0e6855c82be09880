"""The operators strung together as a block uses them: ExpertBlock's gradients against torch.autograd
in float64, routing by scores in ExpertLayer, a padded batch, a captured step, and FP8 serving."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.training import ExpertBlock, ExpertLayer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def make(M, H, I, E, k, seed, **how):
    g = gen(seed)
    b = ExpertBlock(M, H, I, E, k, generator=g, **how)
    b.w_pre.copy_(1 + 0.2 * torch.randn(H, device="cuda", generator=g))
    b.w_post.copy_(1 + 0.2 * torch.randn(H, device="cuda", generator=g))
    if b.gate is not None:
        b.gate.copy_(0.5 + 0.2 * torch.randn(H, device="cuda", generator=g))
    if b.layer.bias is not None:
        b.layer.bias.copy_(0.05 * torch.randn(E, device="cuda", generator=g))
    return b, torch.randn(M, H, device="cuda", generator=g).to(BF16), torch.randn(M, H, device="cuda", generator=g).to(BF16)


def reference(b, x, dout, live):
    """out, dx and the parameters' gradients by autograd in float64, with the block's choice of experts."""
    n = live
    xd = x[:n].double().requires_grad_()
    p = {k: v.double().requires_grad_() for k, v in b.params.items()}
    w13, w2 = b.layer.w13.double().requires_grad_(), b.layer.w2.double().requires_grad_()

    def norm(v, w):
        return v / (v.square().mean(1, keepdim=True) + b.eps).sqrt() * w

    z = norm(xd, p["w_pre"])
    logits = z @ p["w_router"].t()
    how = b.layer.scores
    s = torch.sigmoid(logits) if how["score"] == L.SCORE_SIGMOID else torch.softmax(logits, 1)
    ids = b.layer.topk_ids[:n].long()
    wt = s.gather(1, ids)
    if how.get("renormalize", True):
        wt = wt / wt.sum(1, keepdim=True)
    wt = wt * how.get("routed_scale", 1.0)
    y = torch.zeros(n, b.H, dtype=torch.float64, device="cuda")
    for e in range(b.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = (z[t] @ w13[e].t()).chunk(2, dim=1)
            y = y.index_add(0, t, (torch.nn.functional.silu(gate) * up * wt[t, j][:, None]) @ w2[e].t())
    u = norm(y, p["w_post"])
    out = b.residual_scale * xd + (u if b.gate is None else p["gate"] * u)
    out.backward(dout[:n].double())
    return out.detach(), xd.grad, {k: v.grad for k, v in p.items()}, (w13.grad, w2.grad)


@pytest.mark.parametrize("M,H,I,E,k,live,how", [
    (96, 128, 64, 8, 2, 96, {}),
    (301, 264, 136, 24, 5, 301, {"scores": {"score": L.SCORE_SIGMOID, "groups": 4, "topk_groups": 2, "group_score": L.GROUP_TOP2,
                                           "routed_scale": 2.5, "balance": True}, "residual_scale": 0.5}),
    (120, 256, 64, 12, 3, 77, {"scores": {"score": L.SCORE_SOFTMAX, "renormalize": False}, "gate_init": None}),
])
def test_block_gradients_match_autograd(M, H, I, E, k, live, how):
    b, x, dout = make(M, H, I, E, k, M, **how)
    n = None if live == M else torch.tensor([live], dtype=torch.int32, device="cuda")
    if n is not None:
        x[live:], dout[live:] = float("nan"), float("nan")       # what padding rows hold has no influence
    out = b.forward(x, n)[:live].clone()
    dx = b.backward(dout)[:live]
    torch.cuda.synchronize()
    assert (b.layer.topk_ids[live:] == -1).all() and (b.layer.topk_ids[:live] >= 0).all()
    want, want_dx, grads, experts = reference(b, x, dout, live)
    # every value passes at most eight BF16 roundings on its way (u = 2^-8, of random sign), z's of
    # which the experts' gradients, the router's and the norms' see through one another: twice that
    tol = 2 * 8 ** 0.5 / 256 / 3 ** 0.5 * 1.5
    assert rel(out, want) < tol and rel(dx, want_dx) < tol
    for name, g in grads.items():
        assert rel(b.grads[name], g) < tol, name
    assert rel(b.layer.grads[0], experts[0]) < tol and rel(b.layer.grads[1], experts[1]) < tol
    assert int(b.layer.status.item()) == 0
    before = {k_: v.clone() for k_, v in b.params.items()}
    b.step(1e-3, balance_rate=1e-2 if b.layer.bias is not None else 0.0)
    torch.cuda.synchronize()
    assert all(not torch.equal(before[k_], v) for k_, v in b.params.items())


def test_block_refusals():
    b, x, dout = make(16, 128, 64, 4, 2, 1)
    with pytest.raises(RuntimeError):
        b.backward(dout)
    with pytest.raises(ValueError):
        b.forward(x[:8])
    with pytest.raises(ValueError):
        b.forward(x.float())
    b.forward(x)
    with pytest.raises(ValueError):
        b.backward(dout.float())
    plain = ExpertLayer(16, 128, 64, 4, 2)
    with pytest.raises(RuntimeError):
        plain.balance(0.1)
    with pytest.raises(RuntimeError):
        plain.route_backward(plain.dweights)
    with pytest.raises(ValueError):
        plain.route(torch.zeros(16, 4, device="cuda"), num_tokens=torch.ones(1, dtype=torch.int32, device="cuda"))


def test_balance_needs_a_route():
    layer = ExpertLayer(16, 128, 64, 4, 2, scores={"score": L.SCORE_SIGMOID, "balance": True})
    with pytest.raises(RuntimeError):
        layer.balance(0.1)                         # (the loads are not there yet)
    assert (layer.bias == 0).all()


def test_block_keeps_passes_apart():
    """A served batch ends what backward may use, and the block's own buffers are no inputs."""
    b, x, dout = make(16, 128, 128, 4, 2, 5)
    b.forward(x)
    b.serve(x)
    with pytest.raises(RuntimeError):
        b.backward(dout)
    for t in (b.out, b.z):
        with pytest.raises(ValueError):
            b.forward(t)
    b.forward(x)
    for t in (b.dx, b.dr, b.dy):
        with pytest.raises(ValueError):
            b.backward(t)
    b.backward(dout)


def test_skipped_steps_do_not_count():
    """The block's parameters after a skipped step and a counted one: those of the counted one alone, bit for bit."""
    results = []
    for skipped in (False, True):
        b, x, dout = make(16, 128, 64, 4, 2, 6)
        b.forward(x)
        b.backward(dout)
        if skipped:
            before = {k: v.clone() for k, v in b.params.items()}
            b.step(1e-2, skip=torch.ones(1, dtype=torch.int32, device="cuda"))
            assert all(torch.equal(before[k], v) for k, v in b.params.items())
        b.step(1e-2)
        torch.cuda.synchronize()
        assert b.steps == 1
        results.append({k: v.clone() for k, v in b.params.items()})
    assert all(torch.equal(results[0][k], v) for k, v in results[1].items())


def test_plain_router_has_a_gradient_too():
    """The softmax over the chosen logits: moe_route_topk's weights, renormalised."""
    layer = ExpertLayer(50, 128, 64, 9, 3, generator=gen(3))
    l = torch.randn(50, 9, device="cuda", generator=gen(4))
    dw = torch.randn(50, 3, device="cuda", generator=gen(5))
    layer.route(l)
    ld = l.double().requires_grad_()
    torch.softmax(ld.gather(1, layer.topk_ids.long()), 1).backward(dw.double())
    # (32 units of 2^-24 of the terms, which are below |dw| < 5)
    assert (layer.route_backward(dw).double() - ld.grad).abs().max() < 5 * 32 * 2.0 ** -24


def test_balance_evens_the_load():
    """Experts of unequal popularity: the bias's steps bring the busiest expert's load down to near its share."""
    M, E, k = 2048, 16, 2
    layer = ExpertLayer(M, 128, 64, E, k, scores={"score": L.SCORE_SIGMOID, "balance": True}, generator=gen(6))
    popular = torch.randn(E, device="cuda", generator=gen(7))
    logits = torch.randn(M, E, device="cuda", generator=gen(8)) + popular
    layer.route(logits)
    first = int(layer.group_rows.max())
    for _ in range(60):
        layer.route(logits)
        layer.balance(0.01)
    layer.route(logits)
    last = int(layer.group_rows.max())
    # (a step of 0.01 in scores that vary by 0.2 moves some 5% of a share)
    assert int(layer.group_rows.sum()) == M * k and last < 1.3 * M * k / E < first


def test_captured_step_repeats_the_eager_one():
    """Forward and backward pass captured into a graph; its replay follows the batch's length."""
    M, H = 64, 256
    b, x, dout = make(M, H, 128, 8, 2, 11)
    n = torch.tensor([M], dtype=torch.int32, device="cuda")
    b.forward(x, n)
    b.backward(dout)
    torch.cuda.synchronize()
    want = [t.clone() for t in (b.out, b.dx, *b.grads.values(), *b.layer.grads)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.forward(x, n)
        b.backward(dout)
    for t in (b.out, b.dx, *b.grads.values(), *b.layer.grads):
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    for a, w in zip((b.out, b.dx, *b.grads.values(), *b.layer.grads), want):
        assert torch.equal(a, w)
    # (the eager pass of the shorter batch, not its rows of the longer one: how many rows an expert
    # has decides between two paths of the grouped products, whose sums run in different orders)
    n.fill_(40)
    b.forward(x, n)
    b.backward(dout)
    torch.cuda.synchronize()
    short = [t.clone() for t in (b.out[:40], b.dx, *b.grads.values(), *b.layer.grads)]
    g.replay()
    torch.cuda.synchronize()
    for a, w in zip((b.out[:40], b.dx, *b.grads.values(), *b.layer.grads), short):
        assert torch.equal(a, w)
    assert (b.layer.topk_ids[40:] == -1).all() and (b.dx[40:] == 0).all()


@pytest.mark.parametrize("M,k", [(1, 2), (100, 4)])
def test_serving_in_fp8(M, k):
    b, x, _ = make(M, 256, 128, 16, k, 20 + M, scores={"score": L.SCORE_SIGMOID, "groups": 4, "topk_groups": 2,
                                                       "group_score": L.GROUP_TOP2, "routed_scale": 1.5, "balance": True})
    trained = b.forward(x).clone()
    served = b.serve(x).clone()
    torch.cuda.synchronize()
    # E4M3 weights and activations: a few percent of the branch, which the norm keeps at the stream's size
    assert rel(served, trained.double()) < 0.1 and int(b.layer.status.item()) == 0
    again = b.serve(x)
    assert torch.equal(again, served)
    b.forward(x)
    b.backward(x)
    b.step(1e-2)
    assert rel(b.serve(x), b.forward(x).double()) < 0.1      # (the new weights, not the old ones)
