"""Pins of the block oracle: choices counted out by hand, gradients against differences."""

import numpy as np
import pytest

from oracle import block as B


def test_choice_by_hand():
    l = np.array([[0.0, 2.0, 1.0, 2.0, -1.0, 3.0]])
    ids, w = B.route_scores(l, 3, score=B.SOFTMAX)
    assert ids.tolist() == [[5, 1, 3]]
    np.testing.assert_allclose(w, [np.exp([3, 2, 2]) / np.exp([3, 2, 2]).sum()])
    # a bias changes the choice and not the scores
    ids, w = B.route_scores(l, 2, bias=np.array([1.0, 0, 0, 0, 0, 0]), renormalize=False, routed_scale=2.0)
    assert ids.tolist() == [[0, 5]]
    np.testing.assert_allclose(w, [[2 / (1 + 1), 2 / (1 + np.exp(-3))]])
    # groups of two: the largest alone says 2, the sum of two says 0
    l = np.array([[1.0, 1.1, 0.0, -9.0, 2.0, -9.0]])
    assert B.route_scores(l, 1, groups=3, topk_groups=1)[0].tolist() == [[4]]
    assert B.route_scores(l, 1, groups=3, topk_groups=1, group_score=B.GROUP_TOP2)[0].tolist() == [[1]]


def test_left_out_experts_and_padding():
    l = np.full((3, 4), -np.inf)
    l[0, 2] = 1.0
    ids, w = B.route_scores(l, 2)
    assert ids.tolist() == [[2, -1], [-1, -1], [-1, -1]] and w[0, 0] == 1.0 and w.sum() == 1.0
    ids, w = B.route_scores(np.zeros((3, 4)), 2, live=1)
    assert ids.tolist() == [[0, 1], [-1, -1], [-1, -1]] and w[1:].sum() == 0
    # tiny scores still share out
    _, w = B.route_scores(np.array([[-900.0, -901.0, -5000.0]]), 2)
    np.testing.assert_allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]])


@pytest.mark.parametrize("score", [B.SOFTMAX, B.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    l, dw = rng.standard_normal((5, 9)), rng.standard_normal((5, 3))
    ids, _ = B.route_scores(l, 3, score=score)
    got, mag = B.route_scores_backward(l, ids, dw, score, renorm, 1.7)

    def value(x):
        w = np.stack([B.scores(row, score)[i] for row, i in zip(x, ids)])
        return (1.7 * dw * (w / w.sum(1, keepdims=True) if renorm else w)).sum()

    for t, e in np.ndindex(l.shape):
        d = np.zeros_like(l)
        d[t, e] = 1e-5
        assert abs((value(l + d) - value(l - d)) / 2e-5 - got[t, e]) < 1e-9
    assert (np.abs(got) <= mag * (1 + 1e-12) + 1e-18).all()


def test_balance():
    assert B.route_balance(np.array([1, 3, 2]), np.zeros(3), 0.5).tolist() == [0.5, -0.5, 0.0]


@pytest.mark.parametrize("post,pre,gate", [(True, True, "channel"), (True, True, "token"), (False, True, "full"), (True, False, "none"),
                                           (False, True, "none")])
def test_norm_gradient_against_differences(post, pre, gate):
    rng = np.random.default_rng(2)
    M, H = 4, 6
    v = {"y": rng.standard_normal((M, H)), "r": rng.standard_normal((M, H)), "w_post": rng.standard_normal(H), "w_pre": rng.standard_normal(H)}
    shape = {"channel": H, "token": (M, 1), "full": (M, H)}
    if gate != "none":
        v["gate"] = rng.standard_normal(shape[gate])
    dh, dz = rng.standard_normal((2, M, H))
    how = {"post_norm": post, "weight_offset": 0.5, "eps": 1e-2}

    def run(x):
        return B.norm_residual(x["y"], x["r"], x.get("gate"), x["w_post"] if post else None, x["w_pre"], residual_scale=0.7, **how)

    def value(x):
        o = run(x)
        return (o["h"] * dh).sum() + ((o["z"] * dz).sum() if pre else 0)

    got = B.norm_residual_backward(v["y"], dh, dz if pre else None, run(v)["h"], v.get("gate"), v["w_post"] if post else None, v["w_pre"],
                                   residual_scale=0.7, **how)
    full = got["dgate_full"]
    grads = {"y": got["dy"], "r": got["dr"], "w_post": got.get("dw_post"), "w_pre": got.get("dw_pre"),
             "gate": {"channel": full.sum(0), "token": full.sum(1, keepdims=True), "full": full, "none": None}[gate]}
    for name, g in grads.items():
        if g is None or name not in v:
            continue
        for i in np.ndindex(v[name].shape):
            x = {k: a.copy() for k, a in v.items()}
            x[name][i] += 1e-5
            up = value(x)
            x[name][i] -= 2e-5
            assert abs((up - value(x)) / 2e-5 - g[i]) < 1e-8 * (1 + abs(g[i])), (name, i)
