"""Serving follows the weights however they change: steps of the layer itself, weights copied in, captured passes."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from tests.test_gpu_block_layer import make

pytestmark = pytest.mark.gpu
SIZES = (24, 256, 128, 8, 2)


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def trained(serve_first, step, seed=31):
    """A block after a pass and a step, with or without having served the old weights."""
    b, x, dout = make(*SIZES, seed)
    if serve_first:
        b.serve(x)
    b.forward(x)
    b.backward(dout)
    step(b)
    return b, x


@pytest.mark.parametrize("how", ["block", "layer"])
def test_serving_after_a_step(how):
    step = (lambda b: b.step(5e-2)) if how == "block" else (lambda b: b.layer.step(5e-2))
    b, x = trained(False, step)
    want = b.serve(x).clone()
    old, _ = trained(True, lambda b: None)
    assert not torch.equal(old.serve(x), want)
    b, x = trained(True, step)
    assert torch.equal(b.serve(x), want)
    assert torch.equal(b.serve(x), want)


def test_serving_copied_weights():
    """As a checkpoint brings them: into the layer's own tensors."""
    other, x = trained(False, lambda b: b.step(5e-2))
    want = other.serve(x).clone()
    b, _, _ = make(*SIZES, 32)
    b.serve(x)
    for mine, its in ((b.layer.models, other.layer.models), (b.layer.params, other.layer.params),
                      (list(b.params.values()), list(other.params.values())), ([b.layer.bias], [other.layer.bias])):
        for t, s in zip(mine, its):
            t.copy_(s)
    assert torch.equal(b.serve(x), want)


def test_captured_serving():
    """A captured pass reads the codes where they lie, so that replays see those of a later pass outside the graph."""
    b, x = trained(True, lambda b: None)
    old = b.serve(x).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.serve(x)
    b.out.zero_()
    g.replay()
    assert torch.equal(b.out, old)
    b.forward(x)
    b.backward(x)
    b.step(5e-2)
    new = b.serve(x).clone()
    junk = torch.full((64 << 20,), 77, dtype=torch.uint8, device="cuda")      # (what was freed would be overwritten)
    b.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, new) and not torch.equal(new, old) and junk[0] == 77


def test_weights_that_change_before_a_captured_pass():
    """The graph forms the codes itself; the next pass outside it forms its own, replayed or not."""
    b, x = trained(False, lambda b: b.layer.step(5e-2))
    want = b.serve(x).clone()
    b, x = trained(True, lambda b: b.layer.step(5e-2))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.serve(x)
    assert torch.equal(b.serve(x), want)
    b.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want)


def test_first_pass_captured():
    """A graph captured before anything was served has its own buffers; a pass outside it has others."""
    b, x = trained(False, lambda b: None)
    other, _ = trained(False, lambda b: None)
    want = other.serve(x).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.serve(x)
    assert torch.equal(b.serve(x), want)                 # (the graph has not run yet)
    for _ in range(2):
        b.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)
    assert int(b.layer.status.item()) == 0


def test_refresh():
    """Writes that leave no trace on the host are seen after refresh."""
    b, x = trained(True, lambda b: None)
    other, _ = trained(False, lambda b: None)
    other.layer.models[0].mul_(1.5)
    want = other.serve(x).clone()
    b.layer.models[0].data.mul_(1.5)
    b.refresh()
    assert torch.equal(b.serve(x), want)
