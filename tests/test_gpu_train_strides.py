"""Row buffers as users' programs have them: single rows of any stride, columns
of a wider buffer beside one another."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from tests.test_gpu_train import BF16, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def test_single_rows_of_any_stride():
    g = gen(3)
    K, N = 64, 48
    s, r = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    w = torch.randn(1, N, K, device="cuda", generator=g).to(BF16)
    dense = torch.randn(1, K, device="cuda", generator=g).to(BF16)
    outs = []
    for column in (False, True):
        def new(width, fill=None):
            t = torch.zeros(width, dtype=BF16, device="cuda") if fill is None else fill.reshape(-1).clone()
            return t.view(width, 1).t() if column else t.view(1, width)

        x, y, dx, xs, out = new(K, dense), new(N), new(K), new(K), new(K)
        dw = torch.zeros(1, N, K, dtype=BF16, device="cuda")
        L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r))
        L.moe_grouped_gemm(L.make_grouped_args(y, w, dx, s, r, input_gradient=True))
        L.moe_grouped_wgrad(L.make_grouped_wgrad_args(y, x, dw, s, r))
        L.moe_gather_rows(x, xs, s, 1)
        L.moe_sum_routes(xs, out, s, 1)
        assert torch.equal(xs, dense) and torch.equal(out, dense) and (y != 0).any()
        outs.append((y.clone(), dx.clone(), dw))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
