"""GPU parity of the norms around a block and their gradient against the float64 reference.

Tolerances.  A sum over a row adds at most H / threads terms a thread, then five and five by
shuffles: with the products' own roundings under 40 half units of 2^-24 of the sum of
magnitudes for every team here (H <= 16384), so a root is off by half of that and its own two
units, a normed value by 32 * 2^-24 of itself; GAMMA = 2^-18 covers a chain of two norms and
the cubes of roots.  Sums over rows add (rows a CTA, at most M / min(M, 2 * 152) + 8 for
warps) + 40 + 8 terms one after another.  The rounding of an output adds U times its value."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import block as B

pytestmark = pytest.mark.gpu
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, F32: 2.0 ** -140}
GAMMA = 2.0 ** -18
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, err, dtype, what):
    g, bound = f64(got), err + U[dtype] * (np.abs(want) + err) + TINY[dtype]
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.abs(g - want)[bad].max(), bound[bad].min())


def rows(M, H, dtype, gen, pad=0, std=1.0):
    """[M, H] view of wider rows whose other columns are NaN."""
    t = torch.full((M, H + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :H] = torch.randn(M, H, generator=gen, device="cuda") * std
    return t[:, :H]


def make(M, H, dtype, stream, wtype, gate, pad, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = {"y": rows(M, H, dtype, g, pad, 0.5), "r": rows(M, H, stream, g, 2 * pad, 2.0),
         "w_post": torch.randn(H, generator=g, device="cuda").to(wtype), "w_pre": torch.randn(H, generator=g, device="cuda").to(wtype),
         "dh": rows(M, H, stream, g, pad, 0.1), "dz": rows(M, H, dtype, g, 3 * pad, 0.1)}
    v["gate"] = {"none": lambda: None, "channel": lambda: torch.randn(H, generator=g, device="cuda").to(wtype),
                 "token": lambda: torch.randn(M, 1, generator=g, device="cuda"), "full": lambda: rows(M, H, dtype, g, pad)}[gate]()
    return v


def out_rows(M, H, dtype, pad):
    t = torch.full((M, H + pad), 77.0, dtype=dtype, device="cuda")
    return t[:, :H], t


def check_forward(M, H, dtype=BF16, stream=None, wtype=None, gate="none", post=True, residual=0.5, pad=0, live=None, fp8=None, offset=0.0,
                  weights=True, seed=0, z=True, h=True):
    stream, wtype = stream or dtype, wtype or dtype
    v = make(M, H, dtype, stream, wtype, gate, pad, seed)
    r = v["r"] if residual is not None else None
    w_post, w_pre = (v["w_post"] if post and weights else None), (v["w_pre"] if weights else None)
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    ho, hw = out_rows(M, H, stream, pad)
    zo, zw = out_rows(M, H, dtype, 2 * pad)
    q = torch.full((M, H), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if fp8 is not None else None
    qs = torch.full((M, H // 128), 77.0, device="cuda") if fp8 is not None else None
    how = {"post_norm": post, "residual_scale": 1.0 if residual is None else residual, "eps": EPS, "weight_offset": offset}
    L.moe_norm_residual(L.make_norm_residual_args(v["y"], h=ho if h else None, z=zo if z else None, r=r, gate=v["gate"], w_post=w_post,
                                                  w_pre=w_pre, q=q, q_scale=qs, scale_mode=fp8 or 0, num_rows=n, **how))
    torch.cuda.synchronize()
    k = M if live is None else min(max(live, 0), M)
    want = B.norm_residual(f64(v["y"]), f64(r), f64(v["gate"]), f64(w_post), f64(w_pre), **how)
    if h:
        close(ho[:k], want["h"][:k], GAMMA * want["h_mag"][:k], stream, "h")
        assert (hw[k:] == 77).all() and (hw[:, H:] == 77).all()
    if z:
        close(zo[:k], want["z"][:k], GAMMA * want["z_mag"][:k], dtype, "z")
        assert (zw[k:] == 77).all() and (zw[:, H:] == 77).all()
    if fp8 is not None:
        scale, err = B.quantised(want["z"], fp8 == 1), GAMMA * want["z_mag"].reshape(M, -1, 128)
        got = f64(qs)
        biggest = err.max(2) / 448.0
        if fp8 == 1:      # a power of two; where the largest value lies that near to one, either
            near = B.quantised(want["z"] * (1 + 1e-4), True) != B.quantised(want["z"] * (1 - 1e-4), True)
            assert ((got == scale) | near)[:k].all() and (np.log2(got[:k][got[:k] > 0]) % 1 == 0).all()
        else:
            assert (np.abs(got - scale) <= biggest + 2 * U[F32] * scale)[:k].all()
        codes = q.float().double().cpu().numpy().reshape(M, -1, 128)
        have = codes * got[:, :, None]
        # a code is off by half a step: 2^-4 of the value, 2^-10 of the scale among the smallest;
        # and 448 times the scale holds the largest value up to the scale's own rounding
        bound = err + np.maximum(2.0 ** -4 * np.abs(want["z"].reshape(M, -1, 128)), 2.0 ** -10 * got[:, :, None]) * (1 + 2.0 ** -20)
        assert (np.abs(have - want["z"].reshape(M, -1, 128)) <= bound)[:k].all()
        assert (codes[k:] == torch.tensor([0x55], dtype=torch.uint8).view(torch.float8_e4m3fn).float().item()).all() and (got[k:] == 77).all()
    return v, ho, zo


WIDTHS = [(1, 7168), (3, 8), (9, 248), (17, 256), (5, 264), (33, 512), (200, 520), (7, 1160), (19, 4096), (6, 8192), (5, 8200), (3, 16384),
          (2, 12296), (700, 128), (40, 1024)]


@pytest.mark.parametrize("M,H", WIDTHS)
def test_forward_widths(M, H):
    check_forward(M, H, BF16, gate="channel", seed=H, pad=8)
    check_forward(M, H, FP16, F32, F32, gate="none", seed=H + 1)
    check_forward(M, H, F32, gate="token", seed=H + 2, post=False)
    if H % 128 == 0:
        check_forward(M, H, BF16, fp8=0, seed=H + 3)
        check_forward(M, H, FP16, F32, fp8=1, seed=H + 4, post=False)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("dtype,stream,wtype", [(BF16, BF16, BF16), (BF16, F32, F32), (FP16, FP16, F32), (FP16, F32, FP16), (F32, F32, F32)])
def test_forward_variants(gate, dtype, stream, wtype):
    for i, (post, residual) in enumerate(((True, 1.0), (False, 1.0), (True, None), (False, None))):
        for M, H in ((13, 384), (11, 1280)):
            check_forward(M, H, dtype, stream, wtype, gate, post, residual, pad=8 * (i % 2), live=(None, 7, 0, 99)[i], offset=(0.0, 1.0)[i % 2],
                          seed=i, weights=i != 2, z=i != 1, fp8=(None, 0, 1, None)[i])
            check_forward(M, H, dtype, stream, wtype, gate, post, residual, seed=i + 50, h=False)


def test_forward_in_place_zero_rows_and_nan():
    M, H = 21, 640
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    y, r = torch.randn(M, H, generator=g, device="cuda").to(BF16), torch.randn(M, H, generator=g, device="cuda").to(BF16)
    w = torch.randn(H, generator=g, device="cuda").to(BF16)
    y[3], r[3] = 0, 0
    y[5, 7], y[6, 8] = float("nan"), float("inf")
    h, z = torch.empty_like(y), torch.empty_like(y)
    q, qs = torch.empty(M, H, dtype=torch.uint8, device="cuda"), torch.empty(M, H // 128, device="cuda")
    L.moe_norm_residual(L.make_norm_residual_args(y, h=h, z=z, r=r, w_post=w, w_pre=w, q=q, q_scale=qs))
    assert (h[3] == 0).all() and (z[3] == 0).all() and (q[3] == 0).all() and (qs[3] == 0).all()
    for bad in (5, 6):
        assert z[bad].isnan().any()
    # and its group's dequantised values, whichever of them it is
    deq = q.view(torch.float8_e4m3fn).float().view(M, H // 128, 128) * qs[:, :, None]
    for bad in (5, 6):
        assert (deq[bad].isnan().any(1) == z[bad].view(H // 128, 128).isnan().any(1)).all()
    good = [i for i in range(M) if i not in (5, 6)]
    assert not deq[good].isnan().any()
    assert not z[good].isnan().any() and not h[good].isnan().any()
    y2, r2 = y.clone(), r.clone()
    L.moe_norm_residual(L.make_norm_residual_args(y2, h=r2, z=y2, r=r2, w_post=w, w_pre=w))
    torch.cuda.synchronize()
    assert torch.equal(r2.view(torch.int16), h.view(torch.int16)) and torch.equal(y2.view(torch.int16), z.view(torch.int16))


def test_codes_are_the_quantisers():
    """With FP32 rows the codes and scales are those of rounding z itself: as the quantiser forms them from BF16 values that hold z."""
    M, H = 64, 1024
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    # rows of +-2^k: their root mean square and each z are exact powers of two times one factor
    y = (torch.randint(0, 2, (M, H), generator=g, device="cuda") * 2.0 - 1.0) * 2.0 ** torch.randint(-3, 3, (M, 1), generator=g, device="cuda")
    w = 2.0 ** torch.randint(-9, 9, (H,), generator=g, device="cuda").float()
    for mode, quantise in ((0, L.moe_quantize_act_1x128), (1, L.moe_quantize_act_1x128_ue8m0)):
        z, q = torch.empty_like(y), torch.empty(M, H, dtype=torch.uint8, device="cuda")
        qs, q2 = torch.empty(M, H // 128, device="cuda"), torch.empty(M, H, dtype=torch.uint8, device="cuda")
        qs2 = torch.empty_like(qs)
        L.moe_norm_residual(L.make_norm_residual_args(y, z=z, w_pre=w, q=q, q_scale=qs, scale_mode=mode, eps=0.0))
        assert torch.equal(z.to(BF16).float(), z)
        quantise(z.to(BF16).contiguous(), q2, qs2)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(qs, qs2)


def check_backward(M, H, dtype=BF16, stream=None, wtype=None, gate="none", post=True, pre=True, dh=True, pad=0, live=None, offset=0.0, a=0.5,
                   weights=True, seed=0, accumulate=False, h_is_y=False, in_place=False):
    stream, wtype = stream or dtype, wtype or dtype
    v = make(M, H, dtype, stream, wtype, gate, pad, seed)
    w_post, w_pre = (v["w_post"] if post and weights else None), (v["w_pre"] if weights and pre else None)
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    k = M if live is None else min(max(live, 0), M)
    h = None if h_is_y or not pre else v["r"]
    how = {"post_norm": post, "residual_scale": a, "eps": EPS, "weight_offset": offset}
    ins = {"dh": v["dh"] if dh else None, "dz": v["dz"] if pre else None}
    want = B.norm_residual_backward(f64(v["y"])[:k], *(None if t is None else f64(t)[:k] for t in (ins["dh"], ins["dz"], h)),
                                    gate=None if v["gate"] is None else f64(v["gate"])[:k] if gate != "channel" else f64(v["gate"]),
                                    w_post=f64(w_post), w_pre=f64(w_pre), **how)
    dy, dyw = out_rows(M, H, dtype, pad)
    dr, drw = out_rows(M, H, stream, 2 * pad)
    if in_place:
        dy, dr = ins["dz"] if pre else v["y"], ins["dh"] if dh else h
    prior = 3.0
    dwp = torch.full((H,), prior, device="cuda") if pre else None
    dwq = torch.full((H,), prior, device="cuda") if post else None
    dg = {"none": lambda: (None, None), "channel": lambda: (torch.full((H,), prior, device="cuda"), None),
          "token": lambda: (torch.full((M, 1), 77.0, device="cuda"), None), "full": lambda: out_rows(M, H, dtype, pad)}[gate]()
    ws = torch.full((L.moe_norm_residual_workspace_size(M, H),), 0xFF, dtype=torch.uint8, device="cuda")
    L.moe_norm_residual_backward(L.make_norm_residual_backward_args(
        v["y"], h=h, gate=v["gate"], w_post=w_post, w_pre=w_pre, dy=dy, dr=dr, dgate=dg[0], dw_post=dwq, dw_pre=dwp, workspace=ws,
        accumulate=accumulate, num_rows=n, **ins, **how))
    torch.cuda.synchronize()
    close(dy[:k], want["dy"], GAMMA * want["dy_mag"], dtype, "dy")
    close(dr[:k], want["dr"], GAMMA * want["dr_mag"], stream, "dr")
    if not in_place:
        for t in (dyw, drw):
            assert (t[k:] == 77).all() and (t[:, H:] == 77).all()
    chain = (M / min(M, 304) + 8 + 40 + 8) * 2.0 ** -24
    for t, name in ((dwp, "dw_pre"), (dwq, "dw_post")):
        if t is not None:
            base = prior if accumulate else 0.0
            close(t, base + want[name], (GAMMA + chain) * (want[name + "_mag"] + base), F32, name)
    full, mag = want["dgate_full"], want["dgate_full_mag"]
    if gate == "channel":
        base = prior if accumulate else 0.0
        close(dg[0], base + full.sum(0), (GAMMA + chain) * (mag.sum(0) + base), F32, "dgate")
    elif gate == "token":
        close(dg[0][:k], full.sum(1, keepdims=True), GAMMA * mag.sum(1, keepdims=True), F32, "dgate")
        assert (dg[0][k:] == 77).all()
    elif gate == "full":
        close(dg[0][:k], full, GAMMA * mag, dtype, "dgate")
        assert (dg[1][k:] == 77).all() and (dg[1][:, H:] == 77).all()


@pytest.mark.parametrize("M,H", WIDTHS)
def test_backward_widths(M, H):
    check_backward(M, H, BF16, gate="channel", seed=H, pad=8)
    check_backward(M, H, FP16, F32, F32, gate="token", seed=H + 1)
    check_backward(M, H, F32, gate="full", seed=H + 2)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("dtype,stream,wtype", [(BF16, BF16, BF16), (BF16, F32, F32), (FP16, FP16, F32), (FP16, F32, FP16), (F32, F32, F32)])
def test_backward_variants(gate, dtype, stream, wtype):
    for i, (post, pre, dh) in enumerate(((True, True, True), (False, True, True), (True, False, True), (True, True, False), (False, False, True))):
        for M, H in ((13, 384), (611, 40), (11, 1280)):
            check_backward(M, H, dtype, stream, wtype, gate, post, pre, dh, pad=8 * (i % 2), live=(None, 7, 99, 0, 5)[i], offset=(0.0, 1.0)[i % 2],
                           weights=i != 3, seed=i, accumulate=i % 2 == 1, in_place=i == 0)


def test_backward_of_a_plain_norm():
    """No stream: h = y."""
    for dtype, stream in ((BF16, BF16), (FP16, F32), (F32, F32)):
        for M, H in ((9, 256), (30, 2048)):
            check_backward(M, H, dtype, stream, post=False, h_is_y=True, dh=False, a=1.0)
            check_backward(M, H, dtype, stream, post=False, h_is_y=True, a=1.0, in_place=True)


def test_backward_many_rows_and_empty_batches():
    check_backward(5000, 136, BF16, F32, F32, gate="channel")
    check_backward(2000, 1288, FP16, gate="channel", accumulate=True)
    H = 264
    y = torch.empty(0, H, dtype=BF16, device="cuda")
    ws = torch.empty(L.moe_norm_residual_workspace_size(0, H), dtype=torch.uint8, device="cuda")
    for accumulate in (False, True):
        dw = torch.full((H,), 3.0, device="cuda")
        L.moe_norm_residual_backward(L.make_norm_residual_backward_args(y, dh=y, dz=y, h=y, dy=y, dw_pre=dw, workspace=ws, accumulate=accumulate))
        assert (dw == (3.0 if accumulate else 0.0)).all()
    L.moe_norm_residual(L.make_norm_residual_args(y, z=y.clone()))


def test_gradient_against_differences():
    """The FP32 forward's differences in a few directions."""
    M, H = 5, 72
    v = make(M, H, F32, F32, F32, "channel", 0, 3)
    v = {k: t.contiguous() for k, t in v.items()}

    def value(x):
        h, z = torch.empty_like(v["y"]), torch.empty_like(v["y"])
        L.moe_norm_residual(L.make_norm_residual_args(x["y"], h=h, z=z, r=x["r"], gate=x["gate"], w_post=x["w_post"], w_pre=x["w_pre"],
                                                      residual_scale=0.7, eps=1e-2))
        return (h.double() * v["dh"]).sum() + (z.double() * v["dz"]).sum(), h

    grads = {"y": torch.empty_like(v["y"]), "r": torch.empty_like(v["y"]), "gate": torch.empty(H, device="cuda"),
             "w_post": torch.empty(H, device="cuda"), "w_pre": torch.empty(H, device="cuda")}
    ws = torch.empty(L.moe_norm_residual_workspace_size(M, H), dtype=torch.uint8, device="cuda")
    L.moe_norm_residual_backward(L.make_norm_residual_backward_args(
        v["y"], dh=v["dh"], dz=v["dz"], h=value(v)[1], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"], residual_scale=0.7, eps=1e-2,
        dy=grads["y"], dr=grads["r"], dgate=grads["gate"], dw_post=grads["w_post"], dw_pre=grads["w_pre"], workspace=ws))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    for name, g in grads.items():
        d = torch.randn(g.shape, generator=gen, device="cuda")
        step = 2.0 ** -8
        up, down = dict(v), dict(v)
        up[name], down[name] = v[name] + step * d, v[name] - step * d
        slope = (value(up)[0] - value(down)[0]) / (2 * step)
        want = (g.double() * d).sum()
        # the values are sums of M H products rounded to 2^-24 of some units, over 2 step; the third derivative is some units
        scale = (v["dh"].abs().sum() + v["dz"].abs().sum()).double()
        assert (slope - want).abs() <= scale * (2.0 ** -22 * 8 / step / 2 + 8 * step ** 2), name


def test_same_bits_again_on_another_stream_and_in_a_graph():
    M, H = 900, 1024
    v = make(M, H, BF16, F32, F32, "channel", 0, 9)

    def call(stream=None):
        o = {"h": torch.empty(M, H, device="cuda"), "z": torch.empty(M, H, dtype=BF16, device="cuda"), "dy": torch.empty(M, H, dtype=BF16, device="cuda"),
             "dr": torch.empty(M, H, device="cuda"), **{k: torch.empty(H, device="cuda") for k in ("dgate", "dw_post", "dw_pre")}}
        ws = torch.empty(L.moe_norm_residual_workspace_size(M, H), dtype=torch.uint8, device="cuda")
        f = L.make_norm_residual_args(v["y"], h=o["h"], z=o["z"], r=v["r"], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"])
        b = L.make_norm_residual_backward_args(v["y"], dh=v["dh"], dz=v["dz"], h=o["h"], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"],
                                               workspace=ws, **{k: o[k] for k in ("dy", "dr", "dgate", "dw_post", "dw_pre")})
        return o, lambda: (L.moe_norm_residual(f, stream=stream), L.moe_norm_residual_backward(b, stream=stream))

    first, go = call()
    go()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, go = call(side)
    go()
    side.synchronize()
    third, go = call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for o in (other, third):
        assert all(torch.equal(o[k], first[k]) for k in first)
