"""Biases of the type's lowest value: the sums of two of them pass FP32's range, and groups are still told apart."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import block as B
from tests.test_gpu_block_route import check

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


@pytest.mark.parametrize("score", [B.SIGMOID, B.SOFTMAX])
@pytest.mark.parametrize("groups,size", [(4, 4), (8, 32), (5, 20), (20, 96)])
def test_groups_of_lowest_biases(score, groups, size):
    rng = np.random.default_rng(groups)
    E, k = groups * size, min(2 * size - 2, 12)
    l = rng.standard_normal((12, E)).astype(np.float32)
    for usual in range(3):                            # groups without a mask: none, one, two
        bias = np.full((groups, size), LOWEST, np.float32)
        bias[0] = -np.inf
        bias[2] = LOWEST / 2 ** 0.25                  # (sums of two pass the range, too, and are larger)
        for g in range(usual):
            bias[groups - 1 - g] = rng.standard_normal(size) * 0.1
        for keep in (2, 3):
            for pair in (B.GROUP_TOP2, B.GROUP_MAX):
                check(l, k, bias=bias.ravel(), score=score, groups=groups, topk_groups=keep, group_score=pair)
    bias = rng.standard_normal((groups, size)).astype(np.float32) * 0.1
    bias[1, 1:], bias[3, :] = LOWEST, LOWEST          # one expert of a group is left, none of another
    for keep in (1, 2, groups - 1):
        check(l, min(k, keep * size), bias=bias.ravel(), score=score, groups=groups, topk_groups=keep, group_score=B.GROUP_TOP2)
    check(l, k, bias=bias.ravel(), score=score)
    big = -bias                                       # and the highest ones
    check(l, k, bias=big.ravel(), score=score, groups=groups, topk_groups=2, group_score=B.GROUP_TOP2)
