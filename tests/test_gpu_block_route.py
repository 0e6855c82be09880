"""GPU parity of routing by scores, its gradient and the balance step against the float64
reference.

Ids are compared exactly: the reference compares 64-bit values, and so does the kernel.
Weights: a careful score is within (4 + |x| / 2) * 2^-23 of the true one (exponential 2 units,
sum and divide 1, twice; for softmax |x| / 2 for the rounding of x = l - m), a ratio of
two such sums of up to 32 terms within twice that and 5 more.  A plain softmax weight has the
total of E fast exponentials below it: 2 + 1.7 |x| units each, which their sizes exp(-x)
average to at most 3, and half a unit for each of E / 32 + 5 additions."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import block as B

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -148}
UNIT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def device(logits, dtype, pad=0):
    """The logits as a view of wider rows whose other columns are NaN."""
    t = torch.full((logits.shape[0], logits.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :logits.shape[1]] = torch.from_numpy(logits).to(dtype).cuda()
    return t[:, :logits.shape[1]]


def run(lg, k, bias=None, id_dtype=torch.int32, live=None, **how):
    M = lg.shape[0]
    ids = torch.full((M, k), -7, dtype=id_dtype, device="cuda")
    w = torch.full((M, k), float("nan"), device="cuda")
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    L.moe_route_scores(L.make_route_scores_args(lg, ids, w, bias=b, num_tokens=n, **how))
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def check(logits, k, dtype=torch.float32, bias=None, pad=0, id_dtype=torch.int32, live=None, **how):
    lg = device(logits.astype(np.float32), dtype, pad)
    seen = lg.double().cpu().numpy()
    b = None if bias is None else bias.astype(np.float32)
    ids, w = run(lg, k, b, id_dtype, live, **how)
    want_ids, want = B.route_scores(seen, k, bias=b, live=live, **how)
    assert (ids == want_ids).all(), (np.argwhere((ids != want_ids).any(1))[:5].ravel(), logits.shape, k)
    E = seen.shape[1]
    with np.errstate(invalid="ignore"):
        far = np.minimum(np.abs(np.take_along_axis(seen, np.maximum(want_ids, 0), 1) - seen.max(1, keepdims=True)), 200.0)
    if how.get("renormalize", True):
        units = 2 * (4 + far / 2) + 5
    else:
        units = 4 + far / 2 + (E / 64 + 9 if how.get("score", B.SIGMOID) == B.SOFTMAX else 0)
    bad = ~(np.abs(w - want) <= (np.nan_to_num(units) + 1) * UNIT * np.abs(want) + 2.0 ** -140)
    bad &= ~(np.isnan(w) & np.isnan(want))
    assert not bad.any(), (int(bad.sum()), w[bad][:4], want[bad][:4])
    return lg, ids


CASES = [
    # (M, E, top_k, groups, kept groups)
    (1, 288, 8, 8, 4), (5, 257, 9, 1, 1), (300, 512, 10, 8, 4), (64, 2048, 32, 1, 1), (40, 2048, 32, 32, 7), (33, 24, 24, 1, 1),
    (50, 7, 1, 1, 1), (17, 1, 1, 1, 1), (200, 36, 4, 12, 5), (100, 96, 5, 3, 1), (64, 30, 3, 5, 5), (70, 32, 4, 32, 9),
    (513, 64, 6, 2, 1), (20, 1000, 31, 4, 3),
]


@pytest.mark.parametrize("M,E,k,groups,keep", CASES)
def test_choice_and_weights(M, E, k, groups, keep):
    rng = np.random.default_rng(M * 7 + E * 3 + k)
    i = 0
    for score in (B.SIGMOID, B.SOFTMAX):
        for biased in (False, True):
            for pair in ((B.GROUP_MAX, B.GROUP_TOP2) if groups > 1 else (B.GROUP_MAX,)):
                dtype = (torch.float32, torch.bfloat16, torch.float16)[i % 3]
                bias = rng.standard_normal(E) * (0.1 if score == B.SIGMOID else 0.5 / E) if biased else None
                check(rng.standard_normal((M, E)) * 2.0, k, dtype, bias, pad=i % 2, id_dtype=(torch.int32, torch.int64)[i % 2],
                      score=score, groups=groups, topk_groups=keep, group_score=pair, renormalize=i % 4 < 2, routed_scale=1.0 + i)
                i += 1


@pytest.mark.parametrize("kind", ["equal", "few values", "equal biases", "saturated", "huge", "tiny bias steps", "neighbours"])
def test_values_near_or_equal(kind):
    """Ties, values a unit apart, scores that round to 1 or to 0: the order of 64-bit values, then of the index."""
    rng = np.random.default_rng(11)
    M, E, k = 48, 256, 9
    bias = rng.standard_normal(E) * 0.05
    l = rng.standard_normal((M, E))
    if kind == "equal":
        l[:], bias[:] = 0.25, 0.0
    elif kind == "few values":
        l = rng.integers(-2, 3, (M, E)).astype(float)
        bias = rng.integers(-1, 2, E) * 0.125
    elif kind == "equal biases":
        l, bias = np.round(l * 4) / 4, np.full(E, 0.5)
    elif kind == "saturated":
        l = 18.0 + rng.random((M, E))          # (FP32 sigmoids are all 1 from 17 on, 64-bit ones from 37)
        bias[:] = 0.0
    elif kind == "huge":
        l *= 300.0
    elif kind == "tiny bias steps":
        l[:] = 1.0
        bias = rng.permutation(E) * 2.0 ** -26
    else:
        l = np.nextafter(np.float32(1.0), np.float32(2.0)) ** rng.integers(0, 9, (M, E))
        bias = rng.integers(0, 3, E) * 2.0 ** -24
    for score in (B.SIGMOID, B.SOFTMAX):
        for groups, keep in ((1, 1), (8, 3)):
            for renorm in (True, False):
                check(l, k, bias=bias, score=score, groups=groups, topk_groups=keep, group_score=B.GROUP_TOP2, renormalize=renorm)
            check(l, k, score=score, groups=groups, topk_groups=keep, group_score=B.GROUP_MAX)
            check(l, k, score=score, groups=groups, topk_groups=keep, group_score=B.GROUP_TOP2)
            check(l, k, torch.bfloat16, score=score, groups=groups, topk_groups=keep)


@pytest.mark.parametrize("near,keep", [(2, 4), (3, 2), (4, 5), (2, 1), (7, 4)])
@pytest.mark.parametrize("score", [B.SIGMOID, B.SOFTMAX])
def test_some_groups_too_near_to_tell(near, keep, score):
    """`near` groups of eight around the cut whose two largest differ in last places only, the others far above or below."""
    rng = np.random.default_rng(19 + near)
    M, G, size, k = 64, 8, 16, 12
    first = max(keep - 1 - near // 2, 0)                     # the cut lies among the groups first .. first + near - 1
    l = np.zeros((M, G, size), np.float32)
    for t in range(M):
        for rank, g in enumerate(rng.permutation(G)):
            at = rng.permutation(size)
            among = first <= rank < first + near
            top = np.float32(2.0 - 0.25 * (first if among else rank))
            two = np.array([top, top - np.float32(0.0625)])
            if among:
                steps = rng.integers(-2, 3, 2) if t % 2 else np.array([1, -1]) * rng.integers(-2, 3)
                two = two + steps.astype(np.float32) * np.spacing(two)
            l[t, g] = -4.0 - rng.random(size)
            l[t, g, at[:2]] = two
    l = l.reshape(M, G * size)
    bias = rng.integers(-1, 2, size) * 2.0 ** -25
    for b in (None, np.zeros(G * size), np.tile(bias, G), rng.standard_normal(G * size) * 2.0 ** -27):
        check(l, k, bias=b, score=score, groups=G, topk_groups=keep, group_score=B.GROUP_TOP2)
        check(l, k, bias=b, score=score, groups=G, topk_groups=keep, group_score=B.GROUP_MAX, renormalize=False)


@pytest.mark.parametrize("E,groups", [(512, 8), (64, 1), (257, 1)])
def test_bias_off_its_16_bytes(E, groups):
    rng = np.random.default_rng(E)
    lg = device((rng.standard_normal((70, E))).astype(np.float32), torch.float32)
    wide = torch.full((E + 8,), float("nan"), device="cuda")
    ids, w = torch.zeros(70, 6, dtype=torch.int32, device="cuda"), torch.zeros(70, 6, device="cuda")
    for off in (0, 1, 2, 3, 4):
        bias = wide[off:off + E]
        bias.copy_(torch.from_numpy(rng.standard_normal(E) * 0.1))
        L.moe_route_scores(L.make_route_scores_args(lg, ids, w, bias=bias, groups=groups, topk_groups=max(groups // 2, 1)))
        want, _ = B.route_scores(lg.double().cpu().numpy(), 6, bias=bias.cpu().numpy(), groups=groups, topk_groups=max(groups // 2, 1))
        assert (ids.cpu().numpy() == want).all(), off


def test_left_out_experts_empty_rows_and_padding():
    rng = np.random.default_rng(3)
    M, E, k = 40, 60, 5
    l = rng.standard_normal((M, E)) * 3
    for t in range(M):
        l[t, rng.permutation(E)[:2 * t if t < 30 else E - (t - 30)]] = -np.inf     # down to ten, nine .. no experts
    bias = rng.standard_normal(E) * 0.1
    for b in (None, bias, np.where(np.arange(E) % 7 == 0, -np.inf, bias)):
        for score in (B.SIGMOID, B.SOFTMAX):
            for groups, keep, pair in ((1, 1, 0), (6, 2, 0), (6, 2, 1), (30, 8, 1), (20, 19, 1)):
                for renorm in (True, False):
                    check(l, k, bias=b, score=score, groups=groups, topk_groups=keep, group_score=pair, renormalize=renorm)
    for live in (-3, 0, 1, 17, M, M + 9):
        check(rng.standard_normal((M, E)), k, bias=bias, live=live)
    ids, w = run(device(l.astype(np.float32), torch.float32)[:0], k)
    assert ids.shape == (0, k)


def test_nan_and_infinities():
    """A NaN is the largest value and stays in the weights that its score is part of."""
    rng = np.random.default_rng(4)
    M, E, k = 24, 72, 4
    l = rng.standard_normal((M, E))
    l[3, 5], l[3, 50], l[4, 0], l[5, 7] = np.nan, np.nan, np.inf, np.nan
    l[6, :] = np.nan
    l[7, 10:20] = np.inf
    bias = rng.standard_normal(E) * 0.1
    nan_bias = bias.copy()
    nan_bias[9], nan_bias[40] = np.nan, np.inf
    for b in (None, bias, nan_bias):
        for groups, keep, pair in ((1, 1, 0), (8, 3, 0), (8, 3, 1)):
            for renorm in (True, False):
                check(l, k, bias=b, groups=groups, topk_groups=keep, group_score=pair, renormalize=renorm)
    ids, w = run(device(l.astype(np.float32), torch.float32), k, score=B.SOFTMAX)
    assert (np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1]).all() and (ids >= 0).all() and (ids < E).all()
    assert np.isnan(w[[3, 4, 5, 6, 7]]).any(1).all() and not np.isnan(w[8:]).any()


def gradient(seen, ids, dw, score, renorm, dtype, scale, live=None, in_place=False, pad=0):
    M, E = seen.shape
    lg = device(seen, dtype, pad)
    out = lg if in_place else device(np.full((M, E), 7.0), dtype, 3 * pad)
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    L.moe_route_scores_backward(L.make_route_scores_backward_args(lg, ids, dw, out, score=score, renormalize=renorm,
                                                                  routed_scale=scale, num_tokens=n))
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def check_gradient(l, ids, score, renorm, dtype=torch.float32, id_dtype=torch.int32, live=None, in_place=False, pad=0, seed=0):
    rng = np.random.default_rng(seed)
    seen = torch.from_numpy(l.astype(np.float32)).to(dtype).double().numpy()
    dw = torch.from_numpy(rng.standard_normal(ids.shape).astype(np.float32)).cuda()
    got = gradient(seen, torch.from_numpy(ids).to(id_dtype).cuda(), dw, score, renorm, dtype, 2.5, live, in_place, pad)
    want, mag = B.route_scores_backward(seen, ids, dw.double().cpu().numpy(), score, renorm, 2.5, live)
    finite = np.where(np.isfinite(seen), seen, 0.0)
    far = np.minimum(np.abs(finite - finite.max(1, keepdims=True)), 200.0)
    units = 2 * (8 + far) + 16 + (seen.shape[1] / 64 + 9 if score == B.SOFTMAX and not renorm else 0)
    err = units * UNIT * mag
    bad = ~(np.abs(got - want) <= err + U[dtype] * (np.abs(want) + err) + TINY[dtype])
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("M,E,k", [(1, 288, 8), (300, 512, 10), (70, 257, 9), (40, 2048, 32), (33, 24, 24), (5, 1, 1), (9, 3, 7), (64, 96, 5)])
def test_gradient(M, E, k):
    rng = np.random.default_rng(M + E + k)
    l = rng.standard_normal((M, E)) * 2
    ids = np.stack([rng.permutation(max(E, k))[:k] for _ in range(M)])
    ids[ids >= E] = -1                       # (k > E: the rest is unlisted)
    i = 0
    for score in (B.SIGMOID, B.SOFTMAX):
        for renorm in (True, False):
            for dtype in (torch.float32, torch.bfloat16, torch.float16):
                check_gradient(l, ids, score, renorm, dtype, (torch.int32, torch.int64)[i % 2], None if i % 3 else M // 2,
                               in_place=i % 4 == 1, pad=i % 2, seed=i)
                i += 1


def test_gradient_of_repeated_unlisted_and_left_out_experts():
    rng = np.random.default_rng(8)
    M, E, k = 30, 40, 6
    l = rng.standard_normal((M, E))
    ids = rng.integers(0, E, (M, k))
    ids[3], ids[4, 2:], ids[5, 0], ids[6, 1], ids[7] = -1, -1, E, 2 ** 31 - 1, 9
    l[8:12, :] = -np.inf
    l[9, ids[9, 0]] = 1.0
    l[12, ids[12, 3]] = -np.inf
    l[13] -= 400.0                            # scores below FP32's range
    for score in (B.SIGMOID, B.SOFTMAX):
        for renorm in (True, False):
            check_gradient(l, ids, score, renorm, in_place=True)
            check_gradient(l, ids, score, renorm, id_dtype=torch.int64)


@pytest.mark.parametrize("score", [B.SIGMOID, B.SOFTMAX])
def test_one_renormalised_weight_has_no_gradient(score):
    """top_k 1: the weight is the factor itself, whatever the logits; not a rounding is left of its gradient."""
    rng = np.random.default_rng(23)
    l, ids = rng.standard_normal((500, 40)) * 3, rng.integers(0, 40, (500, 1))
    dw = torch.from_numpy(rng.standard_normal((500, 1)).astype(np.float32)).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        got = gradient(l, torch.from_numpy(ids).to(torch.int32).cuda(), dw, score, True, dtype, 2.5)
        assert (got == 0).all()


def test_gradient_against_differences():
    rng = np.random.default_rng(9)
    M, E, k = 6, 20, 4
    l = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32)).cuda()
    ids, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    dw = torch.from_numpy(rng.standard_normal((M, k)).astype(np.float32)).cuda()
    for score in (L.SCORE_SIGMOID, L.SCORE_SOFTMAX):
        for renorm in (True, False):
            L.moe_route_scores(L.make_route_scores_args(l, ids, w, score=score, renormalize=renorm))
            g = torch.empty_like(l)
            L.moe_route_scores_backward(L.make_route_scores_backward_args(l, ids, dw, g, score=score, renormalize=renorm))
            want = ids.clone()
            for e in range(E):
                step = torch.zeros_like(l)
                step[:, e] = 2.0 ** -6
                up, down = torch.empty_like(w), torch.empty_like(w)
                for x, to in ((l + step, up), (l - step, down)):
                    # (by the kept ids: the choice is not differentiated)
                    s = torch.sigmoid(x.double()) if score == L.SCORE_SIGMOID else torch.softmax(x.double(), 1)
                    s = s.gather(1, want.long())
                    to.copy_(s / s.sum(1, keepdim=True) if renorm else s)
                # (a difference is off by the third derivative, below h^2 / 6 times a few, and rounding 2^-24 / h)
                assert ((((up - down) * dw).sum(1) / 2.0 ** -5) - g[:, e]).abs().max() < 1e-3


def test_balance():
    rng = np.random.default_rng(5)
    for E in (1, 3, 31, 257, 1024, 2048):
        load = rng.integers(0, 2 ** 31 - 1 if E == 31 else 50, E).astype(np.int32)
        load[:E // 2] = load[0]
        bias = rng.standard_normal(E).astype(np.float32)
        b, ld = torch.from_numpy(bias).cuda(), torch.from_numpy(load).cuda()
        out = torch.empty_like(b)
        L.moe_route_balance(ld, b, 0.25, out=out)
        want = (bias + np.float32(0.25) * np.sign(load.astype(object).sum() - load.astype(object) * E).astype(np.float32)).astype(np.float32)
        assert (out.cpu().numpy() == want).all() and (b.cpu().numpy() == bias).all()
        L.moe_route_balance(ld, b, 0.25)
        assert (b.cpu().numpy() == want).all()


def test_same_bits_again_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(6)
    M, E, k = 700, 288, 8
    lg = device(rng.standard_normal((M, E)), torch.float32)
    bias = torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).cuda()
    n = torch.tensor([650], dtype=torch.int32, device="cuda")
    outs = [(torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")) for _ in range(3)]
    recs = [L.make_route_scores_args(lg, i, w, bias=bias, groups=8, topk_groups=4, group_score=L.GROUP_TOP2, num_tokens=n) for i, w in outs]
    L.moe_route_scores(recs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.moe_route_scores(recs[1], stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.moe_route_scores(recs[2])
    g.replay()
    torch.cuda.synchronize()
    for i, w in outs[1:]:
        assert torch.equal(i, outs[0][0]) and torch.equal(w, outs[0][1])
    n.fill_(100)                              # a replay follows the batch's length
    g.replay()
    torch.cuda.synchronize()
    assert (outs[2][0][100:] == -1).all() and torch.equal(outs[2][0][:100], outs[0][0][:100])
