"""The training kernels where one launch goes round its loops: more rows, chunks
and tiles than CTAs, and buffers of more than 2^31 elements."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import train as T
from tests import test_gpu_train as G
from tests import test_gpu_train_states as S
from tests.test_gpu_train import BF16, F32, FP16, HYPER, close, f64, gamma, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


# Row kernels: at most 64 CTAs an SM, of 8 rows or 256 vectors each: 77824 rows
# or 2.5 million vectors in a trip on 152 SMs.

def test_gather_of_more_rows_than_a_trip():
    g = gen(1)
    M, k, rows = 70_001, 2, 170_003
    x = torch.randn(M, 24, device="cuda", generator=g).to(BF16)
    ids = torch.randint(-5, M * k + 50, (rows,), device="cuda", generator=g, dtype=torch.int32)
    xs = torch.full((rows, 24), float("nan"), dtype=BF16, device="cuda")
    L.moe_gather_rows(x, xs, ids, k)
    live = (ids >= 0) & (ids < M * k)
    want = torch.where(live[:, None], x[(ids.long() // k).clamp(0, M - 1)], torch.zeros((), dtype=BF16, device="cuda"))
    assert torch.equal(xs, want)


@pytest.mark.parametrize("dtype,vecs", [(BF16, 3), (F32, 1)])
def test_sum_of_more_vectors_than_a_trip(dtype, vecs):
    g = gen(2)
    M, k, rows, width = 5_300_000 // vecs + 1, 2, 4096, vecs * (4 if dtype == F32 else 8)
    y = torch.randn(rows, width, device="cuda", generator=g).to(dtype)
    slot = torch.randint(-1, rows, (M, k), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full((M, width), float("nan"), dtype=dtype, device="cuda")
    L.moe_sum_routes(y, out, slot.view(-1), k)
    wide = torch.cat([y, torch.zeros(1, width, dtype=dtype, device="cuda")])      # (slot -1: a row of zeros)
    want = wide[slot[:, 0].long()].float() + wide[slot[:, 1].long()].float()      # two terms: one rounding in FP32
    assert torch.equal(out, want.to(dtype))


def test_swiglu_gradient_of_more_rows_than_a_trip():
    """Rows repeat every 1000: so do the results."""
    g = gen(3)
    n, times, I = 1000, 170, 16
    tile = lambda t: t.repeat(times, *([1] * (t.dim() - 1)))                      # noqa: E731
    dh, pre = torch.randn(n, I, device="cuda", generator=g).to(BF16), torch.randn(n, 2 * I, device="cuda", generator=g).to(BF16)
    wt = torch.rand(n, device="cuda", generator=g)
    outs = []
    for a, b, w in ((dh, pre, wt), (tile(dh), tile(pre), tile(wt))):
        dpre, h, dw = torch.empty_like(b), torch.empty_like(a), torch.empty_like(w)
        L.moe_swiglu_backward(L.make_swiglu_backward_args(a, b, dpre, h=h, route_weights=w, dweights=dw))
        outs.append((dpre, h, dw))
    for one, many in zip(*outs):
        assert torch.equal(tile(one), many)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_swiglu_products_of_many_tiles_a_pair(dtype):
    """Some 700 tiles on 76 pairs: both accumulators, the queue and the rows of
    route weights go round."""
    counts = [int(n) for n in np.random.default_rng(4).integers(0, 400, 90)]
    G.test_grouped_swiglu_epilogue(counts, 136, 1056, dtype, "routes")


def test_adamw32_over_many_chunks():
    """More chunks than CTAs, against the formula in 64 bits."""
    g = gen(19)
    ts = G._tensors([6_000_001, 3001], 32, F32, BF16, g)
    prior = [(f64(x["param"]), f64(x["grad"]), f64(x["exp_avg"]), f64(x["exp_avg_sq"])) for x in ts]
    S._step(ts)
    e = 2.0 ** -23
    for x, (p, gr, m, v) in zip(ts, prior):
        p1, m1, v1, r1, upd = T.adamw(p, gr, m, v, weight_decay=0.0, **HYPER)
        em = 3 * e * (np.abs(m) + np.abs(gr))
        assert (np.abs(f64(x["exp_avg"]) - m1) <= em).all()
        assert (np.abs(f64(x["exp_avg_sq"]) - v1) <= 5 * e * v1).all()
        err = 2 * e * np.abs(p) + 2 * (upd * 12 * e + HYPER["lr"] * em / (r1 + HYPER["eps"]))
        assert (np.abs(f64(x["param"]) - p1) <= err).all()
        assert torch.equal(x["model"], x["param"].to(BF16))


# ------------------------------------------------------------------ beyond 2^31 elements

def test_products_with_weights_beyond_32_bit_offsets():
    """The last group's weights lie past element 2^31, for tiles and for few slots."""
    g = gen(5)
    E, N, K = 9, 16384, 16384
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    w[E - 1] = (torch.randn(N, K, device="cuda", generator=g) * K ** -0.5).to(BF16)
    cols = torch.randint(0, N, (64,), device="cuda", generator=g)
    cols[0] = N - 1
    for n in (3, 300):
        s = torch.zeros(E, dtype=torch.int32, device="cuda")
        r = torch.zeros(E, dtype=torch.int32, device="cuda")
        r[E - 1] = n
        x = torch.randn(n, K, device="cuda", generator=g).to(BF16)
        y, dx = torch.empty(n, N, dtype=BF16, device="cuda"), torch.empty(n, K, dtype=BF16, device="cuda")
        L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r))
        part = w[E - 1, cols].double()
        mag = f64(x.double().abs() @ part.abs().t())
        close(y[:, cols], f64(x.double() @ part.t()), gamma(K) * mag, BF16, "forward")
        L.moe_grouped_gemm(L.make_grouped_args(x, w, dx, s, r, input_gradient=True))       # x as dy: N = K
        part = w[E - 1][:, cols].double()
        close(dx[:, cols], f64(x.double() @ part), gamma(N) * f64(x.double().abs() @ part.abs()), BF16, "gradient")
        dw = torch.empty(E, N, K, dtype=BF16, device="cuda")
        L.moe_grouped_wgrad(L.make_grouped_wgrad_args(x, x, dw, s, r))
        a = x[:, cols].double()
        close(dw[E - 1, cols], f64(a.t() @ x.double()), gamma(n) * f64(a.abs().t() @ x.double().abs()), BF16, "dw")
        assert not dw[:E - 1].any()
        del dw


def test_rows_beyond_32_bit_offsets():
    """Slots past element 2^31 of their buffers."""
    g = gen(6)
    width, n = 16384, 200
    first = (1 << 31) // width + 8
    rows = first + n
    xs = torch.empty(rows, width, dtype=BF16, device="cuda")
    x = torch.randn(n, width, device="cuda", generator=g).to(BF16)
    ids = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    ids[first:] = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)
    L.moe_gather_rows(x, xs, ids, 1)
    assert torch.equal(xs[first:], x.flip(0)) and not xs[:first].any()
    out = torch.empty_like(x)
    L.moe_sum_routes(xs, out, torch.arange(rows - 1, first - 1, -1, dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(out, x)
    # products and the SwiGLU gradient over the same slots
    s, r = torch.tensor([first], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    w = (torch.randn(1, 64, width, device="cuda", generator=g) * width ** -0.5).to(BF16)
    y = torch.empty(rows, 64, dtype=BF16, device="cuda")
    L.moe_grouped_gemm(L.make_grouped_args(xs, w, y, s, r))
    want, mag = x.flip(0).double() @ w[0].double().t(), x.flip(0).double().abs() @ w[0].double().abs().t()
    close(y[first:], f64(want), gamma(width) * f64(mag), BF16)
    wide = torch.empty(rows, width, dtype=BF16, device="cuda")
    L.moe_grouped_gemm(L.make_grouped_args(y, w, wide, s, r, input_gradient=True))
    dy = y[first:].double()
    close(wide[first:], f64(dy @ w[0].double()), gamma(64) * f64(dy.abs() @ w[0].double().abs()), BF16)
    ids[first:] = torch.arange(n, dtype=torch.int32, device="cuda")
    I = width // 2
    one, many = torch.empty(n, width, dtype=BF16, device="cuda"), wide
    dh = torch.randn(n, I, device="cuda", generator=g).to(BF16)
    L.moe_swiglu_backward(L.make_swiglu_backward_args(dh, x.flip(0).contiguous(), one))
    far = torch.empty(rows, I, dtype=BF16, device="cuda")
    far[first:] = dh
    L.moe_swiglu_backward(L.make_swiglu_backward_args(far, xs, many, route_ids=ids))
    assert torch.equal(many[first:], one)


def test_adamw_beyond_32_bit_offsets(monkeypatch):
    """A tensor of more than 2^31 elements: its last ones as the formula has them."""
    n, tail = (1 << 31) + 5003, 4096 + 5003 % 128
    first = n - tail
    assert first % 128 == 0
    small = G._tensors([tail], 8, BF16, BF16, gen(7))[0]
    big = {k: torch.zeros((n + 127) // 128 if "scale" in k else n, dtype=v.dtype, device="cuda") for k, v in small.items()}
    for k, v in small.items():
        big[k][first // 128 if "scale" in k else first:] = v
    monkeypatch.setattr(S, "_random20", lambda seed, tensor, count: T.hash20(seed, tensor, count, first=first))
    m, r, ms, rs = S._formula32(small, 0, 11, 1.0, **HYPER)
    S._step([big], seed=11)
    for name, codes, scale in (("exp_avg", m, ms), ("exp_avg_sq", r, rs)):
        assert (big[name + "_scale"][first // 128:].cpu().numpy() == scale).all(), name
        assert (f64(big[name][first:].float()) == codes).all(), name
    S._step([small], seed=11)                        # (the parameter does not depend on the seed)
    assert torch.equal(big["param"][first:], small["param"]) and torch.equal(big["model"][first:], small["model"])
    assert not big["param"][:first].any()
