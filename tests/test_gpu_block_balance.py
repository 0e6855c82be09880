"""The balance bias in a block's step: by the loads of the pass that was trained on, and not where the step is left out."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from tests.test_gpu_block_layer import make

pytestmark = pytest.mark.gpu
SIZES = (64, 256, 128, 8, 2)


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def test_a_served_batch_has_no_part_in_the_balance():
    results = []
    for between in ("nothing", "serve", "serve before backward's step"):
        b, x, dout = make(*SIZES, 41)
        other = torch.randn(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(x.dtype)
        b.serve(other)
        b.forward(x)
        load = b.layer.group_rows.clone()
        b.backward(dout)
        if between != "nothing":
            b.serve(other)
            assert not torch.equal(torch.sign(b.layer.group_rows * 8 - 128), torch.sign(load * 8 - 128))
        b.step(1e-3, balance_rate=0.5)
        results.append(b.layer.bias.clone())
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])


def test_a_skipped_step_leaves_the_bias():
    for flag in (1, 0):
        b, x, dout = make(*SIZES, 42)
        b.forward(x)
        b.backward(dout)
        before = b.layer.bias.clone()
        b.step(1e-3, balance_rate=0.5, skip=torch.tensor([flag], dtype=torch.int32, device="cuda"))
        if flag:
            assert torch.equal(b.layer.bias, before)
        else:
            skipped_not = b.layer.bias.clone()
    b, x, dout = make(*SIZES, 42)
    b.forward(x)
    b.backward(dout)
    b.step(1e-3, balance_rate=0.5)
    assert torch.equal(b.layer.bias, skipped_not) and not torch.equal(skipped_not, before)


def test_a_step_that_cannot_balance_changes_nothing():
    b, x, dout = make(*SIZES, 43, scores={"score": L.SCORE_SIGMOID})
    b.forward(x)
    b.backward(dout)
    before = [t.clone() for t in (*b.params.values(), *b.layer.params)]
    with pytest.raises(RuntimeError):
        b.step(1e-2, balance_rate=0.5)                 # (no bias)
    assert all(torch.equal(t, s) for t, s in zip((*b.params.values(), *b.layer.params), before)) and b.steps == 0
    b, x, _ = make(*SIZES, 43)
    b.serve(x)
    with pytest.raises(RuntimeError):
        b.step(1e-2, balance_rate=0.5)                 # (no pass to balance by)
    b.forward(x)
    with pytest.raises(ValueError):
        b.step(1e-2, balance_rate=float("nan"))
    assert b.steps == 0
    b.backward(x)
    b.step(1e-2, balance_rate=None)                    # (as without)
    assert b.steps == 1
