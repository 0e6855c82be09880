"""What ExpertBlock refuses as inputs: buffers that the pass writes while its input is still needed."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from tests.test_gpu_block_layer import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def test_a_pass_does_not_overwrite_its_input():
    M = 16
    b, x, dout = make(M, 128, 128, 4, 2, 1)
    layer = b.layer
    for t in (b.z, b.out, b.dy, b.dr, b.dx, layer.out, layer.dx, layer.xs[:M], layer.ys[:M], layer.dys[:M], b.dr[:].view(M, 128)):
        with pytest.raises(ValueError):
            b.forward(t)
    n = torch.full((1,), M, dtype=torch.int32, device="cuda")
    b.forward(x)
    for call in (b.forward, b.serve):
        for t in (b.z, b.out):
            kept = t.clone()
            with pytest.raises(ValueError):
                call(t, n)
            assert torch.equal(t, kept)              # (refused before anything is written)
    for t in (b.dy, b.dr, b.dx, layer.dx):
        b.forward(x)
        with pytest.raises(ValueError):
            b.backward(t)
    # the output's gradient may be the output itself, and a served input is only read
    b.forward(x)
    want = b.backward(b.out.clone()).clone()
    b.forward(x)
    assert torch.equal(b.backward(b.out), want)
    b.dx.copy_(x)
    served = b.serve(x).clone()
    assert torch.equal(b.serve(b.dx), served)
