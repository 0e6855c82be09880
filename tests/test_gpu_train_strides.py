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


def test_columns_of_one_buffer():
    """Inputs and outputs side by side in wider rows: the results of separate buffers."""
    g = gen(4)
    n, I, K = 300, 64, 64
    a = torch.randn(n, 3 * I, device="cuda", generator=g).to(BF16)
    outs = []
    for beside in (False, True):
        wide = torch.zeros(n, 8 * I, dtype=BF16, device="cuda")
        place = iter(range(0, 8 * I, I))

        def new(width, fill=None):
            if beside:
                at = [next(place) for _ in range(width // I)][0]
                t = wide[:, at:at + width]
            else:
                t = torch.zeros(n, width, dtype=BF16, device="cuda")
            return t if fill is None else t.copy_(fill)

        s = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
        r = torch.tensor([100, 200], dtype=torch.int32, device="cuda")
        w = torch.randn(2, 2 * I, K, device="cuda", generator=gen(5)).to(BF16)
        x, pre, h, dpre, dh = new(K, a[:, :K]), new(2 * I), new(I), new(2 * I), new(I, a[:, K:2 * K])
        L.moe_grouped_gemm(L.make_grouped_args(x, w, h, s, r, epilogue=L.GROUPED_SWIGLU, pre=pre))
        first = h.clone()
        L.moe_swiglu_backward(L.make_swiglu_backward_args(dh, pre, dpre, h=h))
        ids = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()
        xs = new(I)
        L.moe_gather_rows(dh, xs, ids, 1)
        L.moe_sum_routes(xs, x, ids, 1)
        outs.append([t.clone() for t in (first, pre, h, dpre, xs, x)])
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    assert torch.equal(outs[0][5], a[:, K:2 * K]) and (outs[0][3] != 0).any()
