"""Softmax scores whose total is as far off as it gets: one large logit, the others at one distance at which
they weigh most, biases that bring the candidates within a few errors of one another.  Ids as of 64-bit values."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import block as B
from tests.test_gpu_block_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


@pytest.mark.parametrize("E,groups,keep", [(64, 1, 1), (257, 1, 1), (512, 8, 4), (2048, 1, 1), (2040, 17, 3)])
def test_near_scores_below_a_large_total(E, groups, keep):
    rng = np.random.default_rng(E)
    x = np.linspace(0.0, 12.0, 4801)
    far = float(x[(((E - 1) * x) / (np.exp(x) + E - 1)).argmax()])
    for at in (0.0, 40.0, -300.0):
        l = np.full((16, E), at - far, np.float32)
        l += (rng.integers(-3, 4, l.shape) * np.spacing(np.float32(far))).astype(np.float32)
        l[np.arange(16), rng.integers(0, E, 16)] = at
        score = 1.0 / (np.exp(far) + E - 1)                      # of most experts; the large one's is exp(far) of it
        for step in (2.0 ** -23, 2.0 ** -21, 2.0 ** -19):
            bias = (rng.integers(-4, 5, E) * step * score * np.exp(far)).astype(np.float32)
            check(l, 8, bias=bias, score=B.SOFTMAX, groups=groups, topk_groups=keep, group_score=B.GROUP_TOP2)
            bias[::3] += np.float32(score * (np.exp(far) - 1))   # a third of them beside the large one
            check(l, 8, bias=bias, score=B.SOFTMAX, groups=groups, topk_groups=keep, group_score=B.GROUP_MAX)
            check(l, 8, torch.bfloat16, bias=bias, score=B.SOFTMAX)
