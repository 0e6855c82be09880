"""AdamW's states at the edges of FP32."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import train as T
from tests.test_gpu_train import F32, HYPER, _tensors, f64, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def _step(ts, **kw):
    L.moe_adamw_step(L.make_adamw_args(L.AdamWTable(ts), **{**HYPER, **kw}))
    torch.cuda.synchronize()


def _values(t, name):
    """What the stored codes stand for."""
    return f64(t[name].view(torch.float8_e4m3fn).float()) * T.per_element(f64(t[name + "_scale"]), t["param"].numel())


@pytest.mark.parametrize("value", [1e25, float("inf")])
def test_adamw8_an_overflow_leaves_its_neighbours_finite(value):
    """Where v passes FP32 its root is held (1e24) or, with an infinite gradient,
    the largest finite value, so that it decays again; the element's own update
    is m / inf = 0 (inf / inf with the infinite one).  No other element and no
    scale becomes infinite or NaN."""
    n = 300
    t = _tensors([n], 8, F32, None, gen(5))[0]
    hit = np.zeros(n, bool)
    hit[7:200:3] = True
    on = torch.from_numpy(hit).cuda()
    t["grad"][on] = value
    before = t["param"].clone()
    root = min(0.1 * value, np.finfo(np.float32).max)
    for k in range(4):
        _step([t], step=3 + k, seed=k)
        for name in ("exp_avg", "exp_avg_sq"):
            assert torch.isfinite(t[name + "_scale"]).all() and np.isfinite(_values(t, name)).all(), (k, name)
        assert torch.isfinite(t["param"][~on]).all(), k
        if np.isfinite(value):
            assert torch.equal(t["param"][on], before[on])
        # the group's largest: the last code, 448 scales, exact to some roundings of 2^-24
        assert abs(_values(t, "exp_avg_sq")[hit].max() / (root * 0.99 ** (k / 2)) - 1) < 20 * (k + 1) * 2.0 ** -24
        t["grad"] = torch.randn(n, generator=gen(9 + k), device="cuda")


@pytest.mark.parametrize("where", ["among ordinary roots", "among tiny roots", "alone", "all of them"])
def test_adamw8_nan_stays_in_its_element(where):
    """A NaN gradient makes its element's states NaN, as with 32-bit states, and no other's."""
    n = 256
    t = _tensors([n], 8, F32, None, gen(6))[0]
    hit = np.zeros(n, bool)
    hit[9] = hit[131] = True
    if where == "among tiny roots":          # codes below the usual range beside it
        t["exp_avg_sq"].view(torch.uint8)[::2] = 0
        t["grad"][::2] = 1e-9
    elif where == "alone":                   # every other root is zero
        for name in ("exp_avg", "exp_avg_sq"):
            t[name].view(torch.uint8).zero_()
        t["grad"].zero_()
    elif where == "all of them":
        hit[:] = True
    on = torch.from_numpy(hit).cuda()
    t["grad"][on] = float("nan")
    for k in range(2):
        _step([t], step=3 + k, seed=k)
        for name in ("exp_avg", "exp_avg_sq"):
            assert (np.isnan(_values(t, name)) == hit).all(), (k, name)
        assert (np.isnan(f64(t["param"])) == hit).all()
        t["grad"] = torch.randn(n, generator=gen(7), device="cuda")


def test_adamw_small_second_moments_without_eps():
    """eps = 0 and v from the smallest subnormal on: the update follows the
    stored v.  Seven roundings of at most 2^-23 each make the tolerance."""
    n = 1 << 16
    g = gen(13)
    v = (10.0 ** (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * 15 - 45)).float().clamp_(min=2.0 ** -149)
    m = torch.randn(n, generator=g, device="cuda") * v.double().sqrt().float()
    t = {"param": torch.zeros(n, device="cuda"), "grad": torch.zeros(n, device="cuda"), "exp_avg": m, "exp_avg_sq": v}
    _step([t], eps=0.0, beta2=0.9999)
    m1, v1 = f64(t["exp_avg"]), f64(t["exp_avg_sq"])
    live = v1 > 0
    assert live.mean() > 0.9
    b1, b2 = HYPER["beta1"], 0.9999
    want = -HYPER["lr"] / (1 - b1 ** 3) * m1[live] / np.sqrt(v1[live] / (1 - b2 ** 3))
    err = np.abs(f64(t["param"])[live] - want) / np.abs(want).clip(1e-30)
    assert err.max() <= 7 * 2.0 ** -23


def _random20(seed, tensor, n):
    i = np.arange(n, dtype=np.uint64)
    M = np.uint64(0xFFFFFFFF)
    key = np.uint64((seed + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF)
    x = (i * np.uint64(0x9E3779B1) + key) & M
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7FEB352D)) & M
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846CA68B)) & M
    return ((x ^ (x >> np.uint64(16))) >> np.uint64(12)).astype(np.int64)


def _formula32(t, index, seed, gs, beta1, beta2, **_):
    """The states' codes and scales after a step, every operation of the formula
    rounded to FP32 on its own: (m values, r values, m scale, r scale)."""
    f = np.float32
    n = t["param"].numel()
    per = lambda s: np.repeat(s, 128)[:n]                                   # noqa: E731
    state = lambda k: t[k].float().cpu().numpy() * per(t[k + "_scale"].cpu().numpy())   # noqa: E731
    g = t["grad"].float().cpu().numpy() * f(gs)
    m, r = state("exp_avg"), state("exp_avg_sq")
    m = m * f(beta1) + g * f(1 - beta1)
    r = np.sqrt((r * r) * f(beta2) + (g * g) * f(1 - beta2))
    out = []
    for x in (m, r):
        b = np.zeros(-(-n // 128) * 128, f)
        b[:n] = np.abs(x)
        s = b.reshape(-1, 128).max(1) * f(1 / 448)
        with np.errstate(divide="ignore", invalid="ignore"):
            out += [np.where(per(s) > 0, x / per(s), f(0)), s]
    mq, ms, y, rs = out
    u = _random20(seed, index, n)
    # from 2^-6 on a code's spacing is 2^20 units of the FP32 pattern, below it 2^-9
    high = ((y.view(np.uint32).astype(np.int64) + u) >> 20 << 20).astype(np.uint32).view(f)
    low = np.floor(np.maximum(y, f(2.0 ** -9)) * f(512) + u.astype(f) * f(2.0 ** -20)) / f(512)
    code = np.where(y >= f(2.0 ** -6), np.minimum(high, f(448)), low)
    return T.e4m3_nearest(mq.astype(np.float64)), np.where((r > 0) & (per(rs) > 0), code, 0), ms, rs


@pytest.mark.parametrize("grad,eps", [(torch.bfloat16, 1e-6), (F32, 1e-6), (F32, 0.0)])
def test_adamw8_codes_are_those_of_the_formula(grad, eps):
    """Bit for bit, over enough chunks that every CTA takes several (456 or so
    CTAs of 2048 elements), for ordinary and for very small states."""
    g = gen(17)
    ts = _tensors([3_000_077, 5000, 200_000], 8, grad, torch.bfloat16, g)
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        ts[0][name][:4000] *= 1e-4           # (the gradients then decide)
        ts[2][name] *= 2.0 ** -57            # second moments around and below 1e-37
    ts[2]["grad"] = (ts[2]["grad"].double() * 2.0 ** -60).to(grad)
    want = [_formula32(t, i, 3, 0.5, **HYPER) for i, t in enumerate(ts)]
    _step(ts, seed=3, eps=eps, grad_scale=torch.tensor([0.5], device="cuda"))
    for i, (t, (m, r, ms, rs)) in enumerate(zip(ts, want)):
        for name, codes, scale in (("exp_avg", m, ms), ("exp_avg_sq", r, rs)):
            assert (t[name + "_scale"].cpu().numpy() == scale).all(), (i, name)
            got = f64(t[name].float())
            assert (got == codes).all(), (i, name, int((got != codes).sum()))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_arguments_that_do_not_fit_the_table(bits):
    """More chunks than the table has change nothing; other state bits leave the tensors as they are."""
    ts = _tensors([3001, 0, 5000, 0], bits, F32, torch.bfloat16, gen(23))
    copies = [[{k: v.clone() for k, v in t.items()} for t in ts] for _ in range(2)]
    for more, group in ((0, ts), (5000, copies[0])):
        args = L.make_adamw_args(L.AdamWTable(group), seed=1, **HYPER)
        args.chunks += more
        L.moe_adamw_step(args)
    before = [{k: v.clone() for k, v in t.items()} for t in copies[1]]
    args = L.make_adamw_args(L.AdamWTable(copies[1]), seed=1, **HYPER)
    args.state_bits = 40 - bits
    L.moe_adamw_step(args)
    torch.cuda.synchronize()
    for a, b, c, d in zip(ts, copies[0], copies[1], before):
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
            assert torch.equal(c[k].view(torch.uint8), d[k].view(torch.uint8)), k


def test_adamw8_first_moments_of_zero_beside_ordinary_roots():
    """Groups whose first moment has decayed to nothing, some with a NaN gradient or one element alone."""
    n = 128 * 40 + 5
    t = _tensors([n], 8, F32, None, gen(29))[0]
    t["exp_avg"].view(torch.uint8).zero_()
    t["grad"].zero_()
    t["grad"][128 * 7 + 3] = 0.25
    t["grad"][128 * 9 + 4] = 1e-30
    m, r, ms, rs = _formula32(t, 0, 3, 1.0, **HYPER)
    _step([t], seed=3)
    for name, codes, scale in (("exp_avg", m, ms), ("exp_avg_sq", r, rs)):
        assert (t[name + "_scale"].cpu().numpy() == scale).all(), name
        assert (f64(t[name].float()) == codes).all(), name
    assert int((f64(t["exp_avg"].float()) != 0).sum()) == 2
    t["grad"].zero_()
    t["grad"][128 * 5 + 1] = float("nan")
    _step([t], seed=4, step=4)
    for name in ("exp_avg", "exp_avg_sq", "param"):
        bad = torch.isnan(t[name].float()).nonzero().view(-1)
        assert bad.tolist() == [128 * 5 + 1], name
