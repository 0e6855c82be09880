"""Routing by scores with numbers of groups that are no power of two, so that a lane has more than 64
experts: ids as of 64-bit values, and weights.

Weights: a careful score is within (4 + |x| / 2) * 2^-23 of the true one, a ratio of two such sums of up to
32 terms within twice that and 5 more.  A plain softmax weight has below it a total of E fast
exponentials, each off by 2 + 1.7 x units (x: the distance to the largest logit), whose average over the
softmax is at most 2 + 1.7 ln E, and half a unit for each of (places + 5) additions, of 128 places."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from fp8_block_scale_gb300.build import build
from oracle import block as B
from tests.test_gpu_block_route import UNIT, device, run

pytestmark = pytest.mark.gpu
SIZES = [(2046, 9, 3, 2), (2040, 12, 12, 5), (2040, 8, 17, 6), (1161, 7, 9, 4), (2040, 10, 24, 11), (1105, 5, 17, 9), (1920, 32, 20, 3),
         (2046, 8, 31, 30), (1285, 6, 5, 1)]
KINDS = ["any", "ties", "equal", "neighbours", "nan", "left out", "far"]


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def inputs(kind, M, E, groups, rng):
    l, bias = rng.standard_normal((M, E)) * 2.0, rng.standard_normal(E) * 0.05
    if kind == "ties":
        l, bias = rng.integers(-2, 3, (M, E)).astype(float), rng.integers(-1, 2, E) * 0.125
    elif kind == "equal":
        l[:], bias[:] = 0.25, 0.0
    elif kind == "neighbours":
        l = np.nextafter(np.float32(1.0), np.float32(2.0)) ** rng.integers(0, 9, (M, E))
        bias = rng.integers(0, 3, E) * 2.0 ** -24
    elif kind == "nan":
        l[0, E - 1], l[1, 3], l[1, E - 2], l[2, :] = np.nan, np.nan, np.nan, np.nan
        l[3, E // 2], bias[E - 1] = np.inf, np.nan
    elif kind == "left out":
        for t in range(M):
            l[t, rng.permutation(E)[:E - 3 * t]] = -np.inf             # 0, 3, 6 .. experts stay
        bias[::7] = -np.inf
    elif kind == "far":                                                # the best experts are each group's last ones
        at = np.arange(E) % (E // groups) >= E // groups - 2
        l[:, at] += 8.0
    return l.astype(np.float32), bias.astype(np.float32)


def check(logits, bias, k, dtype, **how):
    lg = device(logits, dtype, 3 if how["score"] else 0)
    seen = lg.double().cpu().numpy()
    ids, w = run(lg, k, bias, **how)
    want_ids, want = B.route_scores(seen, k, bias=bias, **how)
    assert (ids == want_ids).all(), (np.argwhere((ids != want_ids).any(1))[:5].ravel(), logits.shape, k, how)
    E = logits.shape[1]
    with np.errstate(invalid="ignore"):
        far = np.abs(np.take_along_axis(seen, np.maximum(want_ids, 0), 1) - np.nanmax(seen, 1, keepdims=True, initial=-np.inf))
    far = np.minimum(np.nan_to_num(far), 200.0)
    units = 2 * (4 + far / 2) + 5 if how["renormalize"] else 4 + far / 2 + (2 + 1.7 * np.log(E) + 133 / 2 if how["score"] == B.SOFTMAX else 0)
    bad = ~(np.abs(w - want) <= (units + 1) * UNIT * np.abs(want) + 2.0 ** -140) & ~(np.isnan(w) & np.isnan(want))
    assert not bad.any(), (int(bad.sum()), w[bad][:4], want[bad][:4], how)


@pytest.mark.parametrize("E,k,groups,keep", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_many_experts_a_lane(E, k, groups, keep, kind, M=9):
    rng = np.random.default_rng(E * 3 + groups)
    logits, bias = inputs(kind, M, E, groups, rng)
    i = 0
    for score in (B.SIGMOID, B.SOFTMAX):
        for b in (None, bias * (1.0 if score == B.SIGMOID else 4.0 / E) if kind not in ("ties", "neighbours") else bias):
            for pair in (B.GROUP_MAX, B.GROUP_TOP2):
                check(logits, b, k, (torch.float32, torch.bfloat16, torch.float16)[i % 3], score=score, groups=groups, topk_groups=keep,
                      group_score=pair, renormalize=i % 4 < 2, routed_scale=1.0 + i)
                i += 1


def test_in_the_bounds_checking_build():
    build(debug_bounds=True)
    with L.use_library(L.LIB_DEBUG_PATH):
        assert L.moe_debug_bounds_enabled()
        L.moe_debug_bounds_read(reset=True)
        for E, k, groups, keep in SIZES[:3]:
            for kind in KINDS:
                test_many_experts_a_lane(E, k, groups, keep, kind, M=4)
        n, f, line = L.moe_debug_bounds_read(reset=True)
        assert n == 0, f"{n} bounds checks failed, first at {f}:{line}"
