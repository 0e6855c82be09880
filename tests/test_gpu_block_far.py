"""Routing and norms over more tokens than a launch has warps, and over rows whose offsets pass 32 bits."""

import pytest
import torch

from fp8_block_scale_gb300 import _lib as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
UNIT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def route(logits, k, bias=None, **how):
    ids = torch.full((logits.shape[0], k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((logits.shape[0], k), float("nan"), device="cuda")
    L.moe_route_scores(L.make_route_scores_args(logits, ids, w, bias=bias, **how))
    return ids, w


def in_64_bits(logits, k, score, bias=None):
    """ids and plain weights; stable sorting keeps the lower of equal indexes first."""
    l = logits.double()
    s = torch.softmax(l, 1) if score == L.SCORE_SOFTMAX else torch.sigmoid(l)
    order = torch.sort(l if bias is None else s + bias.double(), dim=1, descending=True, stable=True).indices[:, :k]
    return order, s.gather(1, order), s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", [L.SCORE_SOFTMAX, L.SCORE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_more_tokens_than_warps(dtype, score, biased):
    M, E, k = 80011, 21, 3
    logits = torch.randn(M, E, device="cuda", generator=gen(1)).to(dtype)
    bias = torch.randn(E, device="cuda", generator=gen(2)) * 0.1 if biased else None
    ids, w = route(logits, k, bias, score=score, renormalize=False)
    want_ids, want, s = in_64_bits(logits, k, score, bias)
    assert torch.equal(ids.long(), want_ids)
    # (a score: exponential, sum and divide, 4 + |x| / 2 units with |x| < 12; the total of a plain softmax 10 more)
    assert ((w.double() - want).abs() <= 21 * UNIT * want).all()
    dw = torch.randn(M, k, device="cuda", generator=gen(3))
    out = torch.full_like(logits, 7.0)
    L.moe_route_scores_backward(L.make_route_scores_backward_args(logits, ids, dw, out, score=score, renormalize=False))
    listed = torch.zeros(M, E, dtype=torch.float64, device="cuda").scatter_(1, want_ids, dw.double())
    mean = (listed * s).sum(1, keepdim=True)
    want = s * (listed - mean) if score == L.SCORE_SOFTMAX else listed * s * (1 - s)
    size = s * (listed.abs() + (listed.abs() * s).sum(1, keepdim=True))       # of its terms
    # (two scores of 21 units and the sum of three products; then one rounding)
    err = 64 * UNIT * size
    assert ((out.double() - want).abs() <= err + torch.finfo(dtype).eps / 2 * (want.abs() + err) + 1e-38).all()


@pytest.mark.parametrize("renormalize", [False, True])
def test_logits_beyond_32_bits(renormalize):
    """Rows 2^30 + 8 elements apart: the last one's offset passes 2^31 elements and 4 GB."""
    E, k, ld = 257, 9, 2 ** 30 + 8
    store = torch.empty(2 * ld + E, dtype=torch.float16, device="cuda")
    far = store.as_strided((3, E), (ld, 1))
    near = torch.randn(3, E, device="cuda", generator=gen(4)).half()
    far.copy_(near)
    dw = torch.randn(3, k, device="cuda", generator=gen(5))
    results = []
    for logits in (near, far):
        ids, w = route(logits, k, score=L.SCORE_SOFTMAX, renormalize=renormalize)
        L.moe_route_scores_backward(L.make_route_scores_backward_args(logits, ids, dw, logits, score=L.SCORE_SOFTMAX,
                                                                      renormalize=renormalize))
        results.append((ids, w, logits.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("ld,rows", [(2 ** 29, 6), (2 ** 31 + 64, 2)])
def test_norm_rows_beyond_32_bits(ld, rows):
    """Rows 1 GB apart, and further apart than 4 GB, against the same rows side by side."""
    H = 256
    store = torch.empty((rows - 1) * ld + H, dtype=BF16, device="cuda")
    far = store.as_strided((rows, H), (ld, 1))
    y = torch.randn(rows, H, device="cuda", generator=gen(6)).to(BF16)
    r = torch.randn(rows, H, device="cuda", generator=gen(7)).to(BF16)
    dz = torch.randn(rows, H, device="cuda", generator=gen(8)).to(BF16)
    w = 1 + 0.1 * torch.randn(H, device="cuda", generator=gen(9))
    workspace = torch.empty(L.moe_norm_residual_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    results = []
    for branch in (y.clone(), far):
        branch.copy_(y)
        h, dr, dw_post, dw_pre = torch.zeros_like(r), torch.zeros_like(r), torch.zeros_like(w), torch.zeros_like(w)
        z = torch.zeros_like(y)
        L.moe_norm_residual(L.make_norm_residual_args(branch, h=h, z=z, r=r, w_post=w, w_pre=w))
        L.moe_norm_residual_backward(L.make_norm_residual_backward_args(branch, h=h, dz=dz, w_post=w, w_pre=w, dy=branch, dr=dr,
                                                                        dw_post=dw_post, dw_pre=dw_pre, workspace=workspace))
        results.append((h, z, branch.clone(), dr, dw_post, dw_pre))
    for a, b in zip(*results):
        # (the sums' order may be another one: 32-bit values within H + 8 units of the largest, 16-bit ones a rounding step more)
        step = 0.0 if a.dtype == F32 else torch.finfo(a.dtype).eps
        assert ((a.double() - b.double()).abs() <= step * a.double().abs() + (H + 8) * UNIT * a.double().abs().max()).all()
