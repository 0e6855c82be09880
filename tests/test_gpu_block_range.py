"""The norms' gradient where roots are far from one: rows of up to 1e17 and of next to nothing.

As test_gpu_block_norm: GAMMA covers the chain of two norms, U the rounding of an output."""

import numpy as np
import pytest
import torch

from fp8_block_scale_gb300 import _lib as L
from oracle import block as B
from tests.test_gpu_block_norm import BF16, F32, GAMMA, close, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _load():
    L.load()


def check(M, H, dtype, stream, size, eps, gate="none", post=True, h_is_y=False, zero=(), seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(t, std):
        return (torch.randn(M, H, generator=g, device="cuda") * std).to(t)

    y, h, dh, dz = rows(dtype, size), rows(stream, size), rows(stream, 1e-2), rows(dtype, 1e-2)
    for t in (y, h):
        t[list(zero)] = 0
    dh = dh * 0 if zero else (dh / size).to(stream)              # (as large as what comes through the norm)
    h = None if h_is_y else h
    w_pre, w_post = 1 + 0.1 * torch.randn(H, generator=g, device="cuda"), 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    gates = {"none": lambda: None, "channel": lambda: 0.5 + torch.rand(H, generator=g, device="cuda"),
             "token": lambda: 0.5 + torch.rand(M, 1, generator=g, device="cuda"), "full": lambda: rows(dtype, 1.0)}
    gate = gates[gate]()
    w_post = w_post if post else None
    how = {"post_norm": post, "residual_scale": 0.5, "eps": eps}
    want = B.norm_residual_backward(f64(y), f64(dh), f64(dz), f64(h), gate=f64(gate), w_post=f64(w_post), w_pre=f64(w_pre), **how)
    dy, dr, dw = torch.empty_like(y), torch.empty(M, H, dtype=stream, device="cuda"), torch.empty(2, H, device="cuda")
    ws = torch.empty(L.moe_norm_residual_workspace_size(M, H), dtype=torch.uint8, device="cuda")
    L.moe_norm_residual_backward(L.make_norm_residual_backward_args(
        y, dh=dh, dz=dz, h=h, gate=gate, w_post=w_post, w_pre=w_pre, dy=dy, dr=dr, dw_post=dw[0] if post else None, dw_pre=dw[1],
        workspace=ws, **how))
    torch.cuda.synchronize()
    close(dr, want["dr"], GAMMA * want["dr_mag"], stream, "dr")
    close(dy, want["dy"], GAMMA * want["dy_mag"], dtype, "dy")
    chain = (8 + 40 + 8) * 2.0 ** -24
    close(dw[1], want["dw_pre"], (GAMMA + chain) * want["dw_pre_mag"], F32, "dw_pre")
    if post:
        close(dw[0], want["dw_post"], (GAMMA + chain) * want["dw_post_mag"], F32, "dw_post")


@pytest.mark.parametrize("size", [1e12, 1e14, 1e16, 1e17])
@pytest.mark.parametrize("dtype,stream", [(BF16, F32), (F32, F32), (BF16, BF16)])
def test_large_rows(size, dtype, stream):
    for i, gate in enumerate(("none", "channel", "token", "full")):
        check(7, 384, dtype, stream, size, 1e-6, gate, seed=i)
        check(5, 384, dtype, stream, size, 1e-6, gate, post=False, seed=i + 9)
    check(5, 1024, dtype, stream, size, 1e-6, post=False, h_is_y=True)
    check(3, 8200, dtype, stream, size, 1e-6, "channel")


@pytest.mark.parametrize("eps", [1e-20, 1e-30, 1e-38])
def test_rows_of_zeros(eps):
    for dtype, stream in ((BF16, F32), (F32, F32)):
        for H, h_is_y in ((384, False), (384, True), (8200, False)):
            check(6, H, dtype, stream, 1.0, eps, post=not h_is_y, h_is_y=h_is_y, zero=(1, 4))


def test_small_rows():
    for size in (1e-9, 1e-14, 1e-16):
        for H, h_is_y in ((384, False), (384, True), (8200, False)):
            check(6, H, F32, F32, size, 0.0, post=not h_is_y, h_is_y=h_is_y)
