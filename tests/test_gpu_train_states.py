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
