"""GPU parity of the training side against the float64 reference.

Tolerances.  A product's 32-bit sum over `depth` terms is off by at most
gamma * (sum of |terms|) with gamma = (depth + 32) * 2^-23: one unit of 2^-23
per addition (the tensor core's additions truncate, which costs up to twice
the 2^-24 of rounding to nearest) and 32 for the roundings inside one
instruction.  The output's rounding adds u * |value|, u = 2^-8 for BF16 and
2^-11 for FP16, and 2^-25 absolute for FP16's subnormals.  The sigmoid is
within (10 + 1.2 |g|) * 2^-23 relatively (documented bounds of the fast
exponential, 2 + 1.173 |g| units, and divide, 2 units, doubled)."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import train as T

pytestmark = pytest.mark.gpu
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, F32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def f64(t):
    return t.double().cpu().numpy()


def gamma(depth):
    return (depth + 32) * 2.0 ** -23


def close(got, want, err, dtype, what=""):
    """|got - rounded want| within `err` (of the value before rounding) and the rounding itself."""
    g, bound = f64(got), err + U[dtype] * (np.abs(want) + err) + TINY[dtype]
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.abs(g - want)[bad].max(), bound[bad].min())


def buffer(rows, width, dtype, gen, pad=0, std=1.0, fill=float("nan")):
    """[rows, width] view of a wider buffer whose other columns hold `fill`."""
    t = torch.full((rows, width + pad), fill, dtype=dtype, device="cuda")
    t[:, :width] = torch.randn(rows, width, generator=gen, device="cuda") * std
    return t[:, :width]


def layout(counts, gap=0, order=None):
    """Starts of groups of `counts` rows with `gap` unused slots before each, in `order`."""
    start = np.zeros(len(counts), np.int64)
    at = gap
    for e in (order if order is not None else range(len(counts))):
        start[e] = at
        at += counts[e] + gap
    return start, at


def groups(counts, gap=0, order=None, empty_start=0):
    start, slots = layout(counts, gap, order)
    start = np.where(np.array(counts) > 0, start, empty_start)
    s = torch.tensor(start, dtype=torch.int32, device="cuda")
    r = torch.tensor(counts, dtype=torch.int32, device="cuda")
    used = np.zeros(slots, bool)
    for _, i in T.spans(start, counts):
        used[i] = True
    return start, s, r, slots, used


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# (rows of each group, K, N): lengths around every tile edge, empty groups,
# single rows, many groups of few rows, inner sizes that fill no tile
SHAPES = [
    ([1], 8, 16),
    ([0, 0, 0], 64, 64),
    ([3, 0, 1, 7], 72, 48),
    ([16, 17, 0, 15], 200, 136),
    ([64, 1, 129], 256, 272),
    ([128, 127], 128, 256),
    ([255, 256, 257, 0, 2], 136, 528),
    ([300], 1160, 712),
    ([513, 40], 64, 144),
    ([1] * 60 + [0] * 20 + [2] * 40, 512, 128),
    ([700, 0, 1, 900], 320, 1024),
]


def test_groups_of_a_plan_match_the_reference():
    rng = np.random.default_rng(5)
    for M, k, E, bm, masked in ((1, 1, 1, 8, 0), (5, 3, 4, 8, 0.3), (700, 6, 96, 64, 0.1), (4096, 8, 288, 16, 0), (3, 2, 5, 8, 1)):
        ids = np.stack([rng.choice(E, k, replace=False) for _ in range(M)]).astype(np.int32)
        ids[rng.random(ids.shape) < masked] = -1
        cap, blocks = L.moe_plan_capacity(M, k, E, bm)
        sorted_ids = torch.randint(-2 ** 31, 2 ** 31 - 1, (cap,), dtype=torch.int32, device="cuda")   # garbage past P
        expert_ids = torch.randint(-2 ** 31, 2 ** 31 - 1, (blocks,), dtype=torch.int32, device="cuda")
        P = torch.empty(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(L.moe_plan_workspace_size(M, k, E), 256), dtype=torch.uint8, device="cuda")
        L.moe_plan(torch.from_numpy(ids).cuda(), E, bm, sorted_ids, expert_ids, P, ws)
        start, rows, slot = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (E, E, M * k))
        L.moe_plan_groups(sorted_ids, expert_ids, P, bm, M * k, start, rows, slot)
        ws_, wr, wslot = T.plan_groups(ids, E, sorted_ids.cpu().numpy(), bm, int(P.item()))
        assert (start.cpu().numpy() == ws_).all() and (rows.cpu().numpy() == wr).all()
        assert (slot.cpu().numpy() == wslot).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_grouped_forward_and_input_gradient(counts, K, N, dtype):
    start, s, r, slots, used = groups(counts, gap=3, order=np.random.default_rng(K).permutation(len(counts)))
    g = gen(K + N)
    w = (torch.randn(len(counts), N, K, generator=g, device="cuda") * 0.2).to(dtype)
    for grad in (False, True):
        a, b = (N, K) if grad else (K, N)
        x = buffer(slots, a, dtype, g, pad=8)
        x[~torch.from_numpy(used).cuda()] = float("nan")
        y = buffer(slots, b, dtype, g, pad=16, fill=7.0)
        before = y.clone()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = L.make_grouped_args(x, w, y, s, r, input_gradient=grad, device_status=st)
        L.moe_grouped_gemm(args)
        ref = T.grouped_input_gradient if grad else T.grouped_forward
        want, mag = ref(f64(x), f64(w), start, counts)
        close(y[used], want[used], gamma(a) * mag[used], dtype, ("gradient" if grad else "forward"))
        assert torch.equal(y[~torch.from_numpy(used)], before[~torch.from_numpy(used)])
        assert (y._base[:, b:] == 7.0).all() and int(st.item()) == 0
        again = y.clone()
        L.moe_grouped_gemm(args)
        assert torch.equal(again[used], y[used])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,K,N", SHAPES)
@pytest.mark.parametrize("kind", ["routes", "slots", "bare"])
def test_grouped_swiglu_epilogue(counts, K, N, dtype, kind):
    start, s, r, slots, used = groups(counts, gap=2)
    g = gen(K * 3 + N)
    w = (torch.randn(len(counts), N, K, generator=g, device="cuda") * K ** -0.5).to(dtype)
    x = buffer(slots, K, dtype, g, pad=8)
    x[~torch.from_numpy(used).cuda()] = float("nan")
    h = buffer(slots, N // 2, dtype, g, pad=8, fill=5.0)
    pre = None if kind == "bare" else buffer(slots, N, dtype, g, pad=8, fill=5.0)
    hb, pb = h.clone(), None if pre is None else pre.clone()
    kw, wt = {}, np.ones(slots)
    if kind == "slots":
        kw["route_weights"] = torch.rand(slots, generator=g, device="cuda")
        wt = f64(kw["route_weights"])
    elif kind == "routes":
        R = max(1, sum(counts))
        ids = np.full(slots, R)
        ids[used] = np.random.default_rng(N).permutation(R)[: used.sum()]
        if used.sum() > 2:
            ids[np.flatnonzero(used)[1]] = R + 5       # an id outside the routes: weight 0
        kw["route_ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        kw["route_weights"] = torch.randn(R, generator=g, device="cuda")
        wt = np.where(ids < R, f64(kw["route_weights"])[np.minimum(ids, R - 1)], 0.0)
    args = L.make_grouped_args(x, w, h, s, r, epilogue=L.GROUPED_SWIGLU, pre=pre, **kw)
    if N % 16:                                         # half rows that fill no 16-byte vector are refused
        with pytest.raises(L.MoeError):
            L.moe_grouped_gemm(args)
        return
    L.moe_grouped_gemm(args)
    want, mag = T.grouped_forward(f64(x), f64(w), start, counts)
    want, mag, wt = want[used], mag[used] * gamma(K), wt[used]
    I = N // 2
    if pre is not None:
        close(pre[used], want, mag, dtype, "pre")
        assert torch.equal(pre[~torch.from_numpy(used)], pb[~torch.from_numpy(used)])
    hw = T.swiglu(want, wt)
    gate, up = want[:, :I], want[:, I:]
    # |silu'| <= 1.1, |silu| <= |g|
    err = np.abs(wt[:, None]) * (1.1 * mag[:, :I] * (np.abs(up) + mag[:, I:]) + (np.abs(gate) + mag[:, :I]) * mag[:, I:])
    err = err + (10 + 1.2 * np.abs(gate)) * 2.0 ** -23 * np.abs(hw)
    close(h[used], hw, err, dtype, "h")
    assert torch.equal(h[~torch.from_numpy(used)], hb[~torch.from_numpy(used)])


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (FP16, FP16), (FP16, F32)])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_grouped_wgrad(counts, K, N, dtype, out):
    start, s, r, slots, used = groups(counts, gap=3, order=np.random.default_rng(K).permutation(len(counts)))
    g = gen(K + 5 * N)
    dy, x = buffer(slots, N, dtype, g, pad=8), buffer(slots, K, dtype, g, pad=16)
    off = ~torch.from_numpy(used).cuda()
    dy[off], x[off] = float("nan"), float("inf")        # neighbours' rows must not count
    dw = torch.full((len(counts), N, K), float("nan"), dtype=out, device="cuda")
    L.moe_grouped_wgrad(L.make_grouped_wgrad_args(dy, x, dw, s, r))
    want, mag = T.grouped_wgrad(f64(dy), f64(x), start, counts)
    err = gamma(max(counts)) * mag
    close(dw, want, err, out, "dw")
    if out == F32:
        base = torch.randn(len(counts), N, K, generator=g, device="cuda")
        acc = base.clone()
        L.moe_grouped_wgrad(L.make_grouped_wgrad_args(dy, x, acc, s, r, accumulate=True))
        close(acc, want + f64(base), err, out, "accumulated")
        empty = np.array(counts) == 0
        assert torch.equal(acc[empty], base[empty])


def test_bad_groups_are_reported_and_skipped():
    g = gen(3)
    for starts, rows in (([0, 60], [4, 5]), ([-1, 8], [4, 4]), ([0, 8], [4, -2])):
        bad = [a < 0 or n < 0 or a + n > 64 for a, n in zip(starts, rows)]
        s, r = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (starts, rows))
        w = torch.randn(2, 64, 32, generator=g, device="cuda").to(BF16)
        x = torch.randn(64, 32, generator=g, device="cuda").to(BF16)
        y = torch.zeros(64, 64, dtype=BF16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r, device_status=st))
        assert int(st.item()) == L.MOE_DEV_BAD_GROUP
        good = np.zeros(64, bool)
        for a, n, b in zip(starts, rows, bad):
            if not b:
                good[a:a + n] = True
        assert (y[~good] == 0).all() and (y[good] != 0).any(1).all()
        st.zero_()
        dw = torch.full((2, 64, 32), 3.0, dtype=BF16, device="cuda")
        L.moe_grouped_wgrad(L.make_grouped_wgrad_args(y, x, dw, s, r, device_status=st))
        assert int(st.item()) == L.MOE_DEV_BAD_GROUP
        for e in range(2):
            assert (dw[e] == 0).all() == bad[e]


def test_infinities_and_nan_follow_the_rows_they_stand_in():
    g = gen(4)
    for K in (64, 512):
        x = torch.randn(40, K, generator=g, device="cuda").to(BF16)
        x[3, 5], x[17, 0] = float("inf"), float("nan")
        w = torch.rand(2, 32, K, generator=g, device="cuda").to(BF16) + 0.5
        y = torch.zeros(40, 32, dtype=BF16, device="cuda")
        s, r = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 20], [20, 20]))
        L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r))
        assert torch.isinf(y[3]).all() and torch.isnan(y[17]).all()
        rest = [i for i in range(40) if i not in (3, 17)]
        assert torch.isfinite(y[rest]).all()


def test_calls_on_another_stream_are_ordered_there():
    g = gen(6)
    x = torch.randn(2048, 256, generator=g, device="cuda").to(BF16)
    w = torch.randn(4, 512, 256, generator=g, device="cuda").to(BF16)
    s = torch.arange(4, dtype=torch.int32, device="cuda") * 512
    r = torch.full((4,), 512, dtype=torch.int32, device="cuda")
    outs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        y = torch.zeros(2048, 512, dtype=BF16, device="cuda")
        dx = torch.zeros(2048, 256, dtype=BF16, device="cuda")
        dw = torch.zeros(4, 512, 256, dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r), stream=stream)
        L.moe_grouped_gemm(L.make_grouped_args(y, w, dx, s, r, input_gradient=True), stream=stream)
        L.moe_grouped_wgrad(L.make_grouped_wgrad_args(y, x, dw, s, r), stream=stream)
        torch.cuda.synchronize()
        outs.append((y, dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_grouped_products_replay_in_a_graph_with_new_groups():
    """The group table is read by the device: a captured graph follows it."""
    g = gen(8)
    x = torch.randn(600, 192, generator=g, device="cuda").to(BF16)
    w = torch.randn(3, 128, 192, generator=g, device="cuda").to(BF16)
    y = torch.zeros(600, 128, dtype=BF16, device="cuda")
    s = torch.tensor([0, 200, 400], dtype=torch.int32, device="cuda")
    r = torch.tensor([200, 200, 200], dtype=torch.int32, device="cuda")
    args = L.make_grouped_args(x, w, y, s, r)
    L.moe_grouped_gemm(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_grouped_gemm(args)
    starts, counts = [500, 0, 3], [100, 1, 450]
    s.copy_(torch.tensor(starts, dtype=torch.int32))
    r.copy_(torch.tensor(counts, dtype=torch.int32))
    y.zero_()
    graph.replay()
    want, mag = T.grouped_forward(f64(x), f64(w), starts, counts)
    used = ~np.isnan(want[:, 0])
    close(y[used], want[used], gamma(192) * mag[used], BF16)
    assert (y[~used] == 0).all()


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("M,k,width", [(1, 1, 8), (5, 3, 24), (300, 9, 264), (70, 10, 2056), (1000, 2, 7168)])
def test_gather_and_sum(M, k, width, dtype):
    rng = np.random.default_rng(M + width)
    g = gen(M)
    slots = M * k + 37
    num = M * k + 20
    ids = rng.permutation(slots)                   # ids >= M * k stand for no route
    ids[0] = -1
    x = buffer(M, width, dtype, g, pad=8)
    xs = buffer(slots, width, dtype, g, pad=16, fill=3.0)
    before = xs.clone()
    rid = torch.tensor(ids, dtype=torch.int32, device="cuda")
    L.moe_gather_rows(x, xs, rid, k, torch.tensor([num], dtype=torch.int32, device="cuda"))
    want = np.zeros((slots, width))
    live = (ids >= 0) & (ids < M * k)
    want[live] = f64(x)[ids[live] // k]
    assert (f64(xs[:num]) == want[:num]).all() and torch.equal(xs[num:], before[num:])
    assert (xs._base[:, width:] == 3.0).all()

    slot = np.full(M * k, -1)
    slot[ids[live]] = np.flatnonzero(live)
    if M > 2:
        slot[k:2 * k] = -1                         # a token whose routes are all masked
        slot[0] = slots                            # outside the buffer
    y = buffer(slots, width, dtype, g, pad=8)
    out = buffer(M, width, dtype, g, pad=8, fill=2.0)
    prior = f64(out)
    for acc in (True, False):
        L.moe_sum_routes(y, out, torch.tensor(slot, dtype=torch.int32, device="cuda"), k, accumulate=acc)
        rows, ok = f64(y), (slot >= 0) & (slot < slots)
        terms = np.where(ok[:, None], rows[np.where(ok, slot, 0)], 0.0).reshape(M, k, width)
        total = terms.sum(1) + (prior if acc else 0.0)
        mag = np.abs(terms).sum(1) + (np.abs(prior) if acc else 0.0)
        close(out, total, (k + 1) * 2.0 ** -24 * mag, dtype, f"sum {acc}")
    if M > 2:
        assert (out[1] == 0).all()
    assert (out._base[:, width:] == 2.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("k", [4, 5, 6, 7, 8, 11, 16, 64])
def test_sum_of_any_number_of_routes(k, dtype):
    test_gather_and_sum(29, k, 136, dtype)


def test_gather_without_tokens_and_sum_without_rows():
    ids = torch.full((16,), 0, dtype=torch.int32, device="cuda")
    xs = torch.full((16, 64), float("nan"), dtype=BF16, device="cuda")
    L.moe_gather_rows(torch.empty(0, 64, dtype=BF16, device="cuda"), xs, ids, 2)
    assert torch.equal(xs, torch.zeros_like(xs))
    out = torch.full((8, 64), float("nan"), dtype=BF16, device="cuda")
    none = torch.empty(0, 64, dtype=BF16, device="cuda")
    L.moe_sum_routes(none, out, ids, 2)
    assert torch.equal(out, torch.zeros_like(out))
    kept = torch.randn(8, 64, device="cuda").to(BF16)
    out.copy_(kept)
    L.moe_sum_routes(none, out, ids, 2, accumulate=True)
    assert torch.equal(out, kept)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,I", [(1, 8), (3, 24), (77, 256), (50, 1032), (2000, 128)])
@pytest.mark.parametrize("kind", ["routes", "slots", "bare", "in place"])
def test_swiglu_backward(rows, I, dtype, kind):
    g = gen(rows + I)
    dh, pre = buffer(rows, I, dtype, g, pad=8, std=0.1), buffer(rows, 2 * I, dtype, g, pad=8, std=2.0)
    pre[0, :8] = torch.tensor([0, 1e4, -1e4, 30, -30, 90, -90, 2.0 ** -14], dtype=dtype)
    dh0, pre0 = f64(dh), f64(pre)
    num, live, ids, kw = rows, np.ones(rows, bool), np.arange(rows), {}
    wt = np.ones(rows)
    if kind in ("slots", "routes"):
        R = rows if kind == "slots" else rows + 3
        kw["route_weights"] = torch.randn(R, generator=g, device="cuda")
        kw["dweights"] = torch.full((R,), 9.0, device="cuda")
        if kind == "routes":
            ids = np.random.default_rng(I).permutation(rows + 6)[:rows]
            live = ids < R
            num = max(1, rows - 2)
            live[num:] = False
            kw["route_ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
            kw["num_rows"] = torch.tensor([num], dtype=torch.int32, device="cuda")
        wt = np.where(live, f64(kw["route_weights"])[np.minimum(ids, R - 1)], 0.0)
    if kind == "in place":
        dpre, h = pre, dh
    else:
        dpre, h = buffer(rows, 2 * I, dtype, g, pad=8, fill=4.0), buffer(rows, I, dtype, g, pad=8, fill=4.0)
    pb, hb = dpre.clone(), h.clone()
    L.moe_swiglu_backward(L.make_swiglu_backward_args(dh, pre, dpre, h=h, **kw))
    want, hw, dwt = T.swiglu_backward(dh0, pre0, wt)
    gate, up = np.abs(pre0[:, :I]), np.abs(pre0[:, I:])
    rel = (10 + 1.2 * np.minimum(gate, 100)) * 2.0 ** -23          # of the sigmoid, and a few products
    sig = T.sigmoid(pre0[:, :I])
    base = np.abs(dh0 * wt[:, None])
    # 1 - sig is off by rel * sig absolutely, times g; the bracket is at most 1 + |g|;
    # below exp(-88) the sigmoid may flush to zero
    eg = base * up * sig * (1 + gate) * 3 * rel + base * up * (1 + gate) * 2.0 ** -120
    eu = base * gate * sig * 2 * rel + base * gate * 2.0 ** -120
    eh = np.abs(wt[:, None]) * gate * up * (sig * 2 * rel + 2.0 ** -120)
    close(dpre[live], want[live], np.concatenate([eg, eu], 1)[live], dtype, "dpre")
    close(h[live], hw[live], eh[live], dtype, "h")
    off = torch.from_numpy(~live)
    assert torch.equal(dpre[off], pb[off]) and torch.equal(h[off], hb[off])
    if "dweights" in kw:
        got = f64(kw["dweights"])
        terms = np.abs(dh0) * gate * sig * up
        err = (terms * (2 * rel + gamma(I))).sum(1)
        assert (np.abs(got[ids[live]] - dwt[live]) <= err[live] + 2.0 ** -24 * np.abs(dwt[live]) + 1e-30).all()
        rest = np.ones(got.size, bool)
        rest[ids[live]] = False
        assert (got[rest] == 9.0).all()


def test_swiglu_backward_without_optional_outputs():
    g = gen(2)
    dh, pre = buffer(9, 16, BF16, g), buffer(9, 32, BF16, g)
    a, b = torch.zeros(9, 32, dtype=BF16, device="cuda"), torch.zeros(9, 32, dtype=BF16, device="cuda")
    h = torch.zeros(9, 16, dtype=BF16, device="cuda")
    L.moe_swiglu_backward(L.make_swiglu_backward_args(dh, pre, a))
    L.moe_swiglu_backward(L.make_swiglu_backward_args(dh, pre, b, h=h))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ AdamW

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, step=3)
SIZES = [1, 3, 127, 128, 129, 4095, 4096, 4097, 20001, 0, 8192]


def _tensors(sizes, bits, grad, model, g, std=1.0):
    out = []
    for n in sizes:
        t = {"param": torch.randn(n, generator=g, device="cuda"),
             "grad": (torch.randn(n, generator=g, device="cuda") * std).to(grad)}
        if model is not None:
            t["model"] = torch.full((n,), -1.0, dtype=model, device="cuda")
        m, r = torch.randn(n, generator=g, device="cuda") * 0.3, torch.rand(n, generator=g, device="cuda") + 1e-4
        if bits == 32:
            t["exp_avg"], t["exp_avg_sq"] = m, r * r
        else:
            for name, v in (("exp_avg", m), ("exp_avg_sq", r)):
                codes = T.e4m3_nearest(f64(v) * 448)     # any codes and any positive scales
                t[name] = torch.from_numpy(codes).float().to(torch.float8_e4m3fn).cuda()
                t[name + "_scale"] = torch.rand(-(-n // 128), generator=g, device="cuda") * 1e-3 + 1e-3
        out.append(t)
    return out


def _before(t, bits):
    n = t["param"].numel()
    if bits == 32:
        return f64(t["exp_avg"]), f64(t["exp_avg_sq"])
    m = f64(t["exp_avg"].float()) * T.per_element(f64(t["exp_avg_scale"]), n)
    return m, (f64(t["exp_avg_sq"].float()) * T.per_element(f64(t["exp_avg_sq_scale"]), n)) ** 2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad,model", [(BF16, BF16), (FP16, FP16), (F32, None)])
def test_adamw_step(bits, grad, model):
    g = gen(bits)
    ts = _tensors(SIZES, bits, grad, model, g)
    ts[2]["weight_decay"] = 0.5
    gs = torch.tensor([0.25], device="cuda")
    prior = [(f64(t["param"]), f64(t["grad"]) * 0.25, *_before(t, bits)) for t in ts]
    table = L.AdamWTable(ts, weight_decay=0.1)
    L.moe_adamw_step(L.make_adamw_args(table, seed=77, grad_scale=gs, **HYPER))
    e = 2.0 ** -23
    for i, (t, (p, gr, m, v)) in enumerate(zip(ts, prior)):
        n = p.size
        if n == 0:
            continue
        wd = 0.5 if i == 2 else 0.1
        p1, m1, v1, r1, upd = T.adamw(p, gr, m, v, weight_decay=wd, **HYPER)
        # sums of two rounded products; the root halves v's error; ten roundings in the update
        em = 3 * e * (np.abs(m) + np.abs(gr))
        erel_v = 5 * e
        eupd = upd * 12 * e + HYPER["lr"] * em / (r1 + HYPER["eps"])
        assert (np.abs(f64(t["param"]) - p1) <= 2 * e * np.abs(p) + 2 * eupd).all(), i
        if model is not None:
            close(t["model"], f64(t["param"]), np.zeros(n), model, "model")
        if bits == 32:
            assert (np.abs(f64(t["exp_avg"]) - m1) <= em).all()
            assert (np.abs(f64(t["exp_avg_sq"]) - v1) <= erel_v * v1).all()
            continue
        for name, x, err in (("exp_avg", m1, em), ("exp_avg_sq", r1, erel_v * r1)):
            scale, codes = f64(t[name + "_scale"]), f64(t[name].float())
            top = T.group_max(x)
            assert (np.abs(scale - top / 448) <= T.group_max(err) / 448 + 2 * e * top / 448).all(), (i, name)
            y = np.abs(x) / T.per_element(scale, n)
            d = err / T.per_element(scale, n) + 4 * e * y        # how far the quotient may be off
            if name == "exp_avg":
                lo, hi = T.e4m3_nearest(np.maximum(y - d, 0)), T.e4m3_nearest(y + d)
                got = np.abs(codes)
                assert (np.sign(codes) * np.sign(x) >= 0).all()
            else:
                u = T.hash20(77, i, n)
                lo, hi = T.e4m3_random(np.maximum(y - d, 0), u), T.e4m3_random(y + d, u)
                # the 20 random bits and the quotient are added in 32 bits: one unit of the last place
                lo, hi = np.minimum(lo, T.e4m3_random(np.maximum(y - d, 0), np.maximum(u - 4, 0))), \
                    np.maximum(hi, T.e4m3_random(y + d, u + 4))
                got = codes
            assert ((got >= lo) & (got <= hi)).all(), (i, name, int(((got < lo) | (got > hi)).sum()))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_second_moment_beyond_fp32(bits):
    # v overflows to infinity, m does not: the update is m / inf = 0
    ts = _tensors([300], bits, F32, None, gen(5))
    ts[0]["grad"][7:200:3] = 1e25
    before = ts[0]["param"].clone()
    L.moe_adamw_step(L.make_adamw_args(L.AdamWTable(ts), seed=1, **HYPER))
    assert torch.equal(ts[0]["param"][7:200:3], before[7:200:3])
    assert bool(torch.isfinite(ts[0]["param"]).all())


def test_adamw_skip_leaves_everything():
    for bits in (32, 8):
        g = gen(9)
        ts = _tensors([300, 5000], bits, F32, BF16, g)
        old = [{k: v.clone() for k, v in t.items()} for t in ts]
        args = L.make_adamw_args(L.AdamWTable(ts), skip=torch.ones(1, dtype=torch.int32, device="cuda"), **HYPER)
        L.moe_adamw_step(args)
        for t, o in zip(ts, old):
            assert all(torch.equal(t[k].view(torch.uint8), o[k].view(torch.uint8)) for k in o)


def test_adamw8_zero_groups_and_lost_roots():
    """A group of zeros stays zero with scale 0; a root far below its group's largest keeps a code."""
    n = 256
    ts = [{"param": torch.ones(n, device="cuda"), "grad": torch.zeros(n, device="cuda"),
           "exp_avg": torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
           "exp_avg_sq": torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
           "exp_avg_scale": torch.zeros(2, device="cuda"), "exp_avg_sq_scale": torch.zeros(2, device="cuda")}]
    ts[0]["grad"][128] = 1.0
    ts[0]["grad"][129] = 1e-12
    table = L.AdamWTable(ts)
    L.moe_adamw_step(L.make_adamw_args(table, **dict(HYPER, step=1)))
    t = ts[0]
    assert t["exp_avg_scale"][0] == 0 and t["exp_avg_sq_scale"][0] == 0
    assert (t["param"][:128] == 1).all()
    assert float(t["exp_avg_sq"].float()[129]) == 2.0 ** -9
    assert float(t["exp_avg_sq"].float()[130]) == 0
    t["grad"].zero_()
    before = t["param"].clone()
    L.moe_adamw_step(L.make_adamw_args(table, **dict(HYPER, step=2)))
    assert float((t["param"] - before).abs().max()) <= 10 * HYPER["lr"]


def test_adamw8_roots_decay_on_average():
    """Under a vanishing gradient the stored roots fall by sqrt(beta2) a step in
    the mean, although each step is far below one code."""
    n, steps = 128 * 200, 40
    g = gen(11)
    r = torch.rand(n, generator=g, device="cuda") * 0.8 + 0.1
    r[::128] = 1.0
    t = {"param": torch.zeros(n, device="cuda"), "grad": torch.zeros(n, device="cuda"),
         "exp_avg": torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
         "exp_avg_scale": torch.zeros(n // 128, device="cuda"),
         "exp_avg_sq": (r * 448).to(torch.float8_e4m3fn), "exp_avg_sq_scale": torch.full((n // 128,), 1 / 448, device="cuda")}
    # the first element of each group is kept at its size by its own gradient
    t["grad"][::128] = 1.0
    old = f64(t["exp_avg_sq"].float()) / 448
    table = L.AdamWTable([t])
    for k in range(steps):
        L.moe_adamw_step(L.make_adamw_args(table, lr=0.0, step=k + 1, beta2=0.999, seed=k))
    new = f64(t["exp_avg_sq"].float()) * np.repeat(f64(t["exp_avg_sq_scale"]), 128)
    keep = np.arange(n) % 128 != 0
    ratio = new[keep].sum() / old[keep].sum()
    # each step's rounding adds noise of at most half a spacing (r / 16), steps and elements independent
    assert abs(ratio - 0.999 ** (steps / 2)) < 6 * np.sqrt(steps) / 16 / np.sqrt(keep.sum())


def test_adamw_in_a_graph_and_with_other_tensors_strides():
    g = gen(12)
    ts = _tensors([1000, 5], 32, BF16, BF16, g)
    ref = [{k: v.clone() for k, v in t.items()} for t in ts]
    args = L.make_adamw_args(L.AdamWTable(ts), **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_adamw_step(args)
    graph.replay()
    L.moe_adamw_step(L.make_adamw_args(L.AdamWTable(ref), **HYPER))
    torch.cuda.synchronize()
    for t, o in zip(ts, ref):
        assert all(torch.equal(t[k], o[k]) for k in o)


@pytest.mark.parametrize("E,per", [(700, 1), (2048, 2), (650, 20), (2048, 0)])
def test_many_groups(E, per):
    """More groups than the few-slots path takes, and the largest table."""
    rng = np.random.default_rng(E + per)
    counts = list(rng.integers(0, 2 * per + 1, E)) if per > 1 else [per] * E
    K, N = 72, 144
    start, s, r, slots, used = groups(counts, gap=1)
    g = gen(E)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 0.2).to(BF16)
    x, y = buffer(slots, K, BF16, g), torch.zeros(slots, N, dtype=BF16, device="cuda")
    dy, dw = buffer(slots, N, BF16, g), torch.full((E, N, K), 9.0, dtype=BF16, device="cuda")
    L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r))
    L.moe_grouped_wgrad(L.make_grouped_wgrad_args(dy, x, dw, s, r))
    want, mag = T.grouped_forward(f64(x), f64(w), start, counts)
    close(y[used], want[used], gamma(K) * mag[used], BF16)
    assert (y[~torch.from_numpy(used)] == 0).all()
    want, mag = T.grouped_wgrad(f64(dy), f64(x), start, counts)
    close(dw, want, gamma(max(counts)) * mag, BF16)


@pytest.mark.parametrize("slots,K,N", [(9, 5000, 320), (16, 1096, 64), (13, 136, 72), (1, 7168, 512), (8, 40, 3088)])
def test_few_slots_with_long_and_short_contractions(slots, K, N):
    """The paths for at most 8 and 16 slots, one and several units side by side."""
    counts = [slots, 0, 1, max(1, slots - 1)]
    start, s, r, rows, used = groups(counts, gap=2)
    g = gen(K)
    w = (torch.randn(4, N, K, generator=g, device="cuda") * K ** -0.5).to(FP16)
    x = buffer(rows, K, FP16, g, pad=8)
    x[~torch.from_numpy(used).cuda()] = float("nan")
    y = torch.zeros(rows, N, dtype=FP16, device="cuda")
    L.moe_grouped_gemm(L.make_grouped_args(x, w, y, s, r))
    want, mag = T.grouped_forward(f64(x), f64(w), start, counts)
    close(y[used], want[used], gamma(K) * mag[used], FP16)
    if N % 16 == 0:
        wt = torch.rand(rows, generator=g, device="cuda")
        h, pre = torch.zeros(rows, N // 2, dtype=FP16, device="cuda"), torch.zeros(rows, N, dtype=FP16, device="cuda")
        L.moe_grouped_gemm(L.make_grouped_args(x, w, h, s, r, epilogue=L.GROUPED_SWIGLU, pre=pre, route_weights=wt))
        assert torch.equal(pre, y)
        hw = T.swiglu(want[used], f64(wt)[used])
        m = gamma(K) * mag[used]
        I = N // 2
        gate, up = np.abs(want[used][:, :I]), np.abs(want[used][:, I:])
        err = 1.1 * m[:, :I] * (up + m[:, I:]) + (gate + m[:, :I]) * m[:, I:] + (10 + 1.2 * gate) * 2.0 ** -23 * np.abs(hw)
        close(h[used], hw, err, FP16)


def test_adamw_with_gradients_of_several_types():
    g = gen(21)
    for bits in (32, 8):
        ts = []
        for grad in (BF16, F32, FP16, BF16):
            ts += _tensors([5000, 77], bits, grad, BF16, g)
        one = [{k: v.clone() for k, v in t.items()} for t in ts]
        L.moe_adamw_step(L.make_adamw_args(L.AdamWTable(ts), seed=5, **HYPER))
        for i, t in enumerate(one):
            # alone, at the same place of its table
            dummy = [dict(t, **{k: v[:0].clone() for k, v in t.items()}) for _ in range(i)]
            L.moe_adamw_step(L.make_adamw_args(L.AdamWTable(dummy + [t]), seed=5, **HYPER))
            for k in t:
                assert torch.equal(t[k].view(torch.uint8), ts[i][k].view(torch.uint8)), (bits, i, k)
