"""Host-side argument checks of routing by scores and of the norms (no GPU needed): the C entry
points and the binding."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

NULL, SHAPE, ALIGN, CAPACITY, DTYPE, OK = 1, 2, 3, 4, 5, 0
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M1 = 1 << 20
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from fp8_block_scale_gb300 import _lib
    from fp8_block_scale_gb300.build import build
    build()
    _lib.load()
    return _lib


def _refused(fn, args, want, **fields):
    old = {k: getattr(args, k) for k in fields}
    for k, v in fields.items():
        setattr(args, k, v)
    got = fn(ctypes.byref(args), None)
    for k, v in old.items():
        setattr(args, k, v)
    assert got == want, (fields, got)


def _route(L):
    a = L.MoeRouteScoresArgs()
    a.logits, a.topk_ids, a.topk_weights, a.bias = M1, 2 * M1, 3 * M1, 4 * M1
    a.M, a.ldlogits, a.E, a.top_k, a.groups, a.topk_groups = 100, 64, 64, 8, 8, 4
    a.dtype, a.id_bits, a.routed_scale = 2, 32, 1.0
    return a


def test_route_scores_refusals(L):
    f, a = L.load().moe_route_scores, _route(L)
    assert f(None, None) == NULL
    for bad in ({"dtype": 3}, {"dtype": -1}, {"id_bits": 16}, {"id_bits": 0}):
        _refused(f, a, DTYPE, **bad)
    for bad in ({"M": -1}, {"M": 1 << 31}, {"M": (1 << 28) + 1, "top_k": 8}, {"E": 0}, {"E": 2049, "ldlogits": 2049}, {"ldlogits": 63},
                {"ldlogits": (1 << 40) + 1}, {"top_k": 0}, {"top_k": -1}, {"top_k": 33}, {"groups": 0}, {"groups": 7}, {"groups": 64},
                {"groups": -8}, {"topk_groups": 0}, {"topk_groups": 9}, {"top_k": 9, "topk_groups": 1}, {"group_score": 2}, {"group_score": -1},
                {"score": 2}, {"score": -1}, {"routed_scale": NAN}, {"routed_scale": INF},
                {"topk_ids": M1 + 4 * 99 * 64}, {"topk_weights": M1}, {"topk_ids": 4 * M1}, {"topk_weights": 2 * M1 + 3196},
                {"num_tokens": 2 * M1}):
        _refused(f, a, SHAPE, **bad)
    for name in ("logits", "topk_ids", "topk_weights"):
        _refused(f, a, NULL, **{name: None})
    for bad in ({"logits": M1 + 2}, {"topk_ids": 2 * M1 + 2}, {"topk_ids": 2 * M1 + 4, "id_bits": 64}, {"topk_weights": 3 * M1 + 1},
                {"bias": 4 * M1 + 2}, {"num_tokens": 5 * M1 + 3}, {"dtype": 0, "logits": M1 + 1}):
        _refused(f, a, ALIGN, **bad)
    _refused(f, a, OK, M=0, logits=None, topk_ids=None, topk_weights=None)


def test_route_scores_backward_refusals(L):
    f = L.load().moe_route_scores_backward
    a = L.MoeRouteScoresBackwardArgs()
    a.logits, a.topk_ids, a.dweights, a.dlogits = M1, 2 * M1, 3 * M1, 4 * M1
    a.M, a.ldlogits, a.lddlogits, a.E, a.top_k, a.dtype, a.id_bits, a.routed_scale = 100, 64, 64, 64, 8, 0, 32, 1.0
    assert f(None, None) == NULL
    for bad in ({"dtype": 4}, {"id_bits": 8}):
        _refused(f, a, DTYPE, **bad)
    for bad in ({"M": -1}, {"E": 0}, {"E": 65}, {"E": 4096, "ldlogits": 4096}, {"lddlogits": 63}, {"lddlogits": (1 << 40) + 1}, {"top_k": 33},
                {"top_k": 0}, {"score": 5}, {"routed_scale": -INF}, {"dlogits": M1 + 2}, {"dlogits": M1, "lddlogits": 72}, {"dlogits": 2 * M1},
                {"dlogits": 3 * M1 - 16}, {"num_tokens": 4 * M1 + 4}):
        _refused(f, a, SHAPE, **bad)
    for name in ("logits", "topk_ids", "dweights", "dlogits"):
        _refused(f, a, NULL, **{name: None})
    for bad in ({"logits": M1 + 1}, {"dlogits": 4 * M1 + 1}, {"topk_ids": 2 * M1 + 1}, {"dweights": 3 * M1 + 2}):
        _refused(f, a, ALIGN, **bad)
    _refused(f, a, OK, M=0)


def test_route_balance_refusals(L):
    f, p = L.load().moe_route_balance, ctypes.c_void_p
    assert f(p(M1), p(2 * M1), p(2 * M1), 0, 1.0, None) == SHAPE and f(p(M1), p(2 * M1), p(2 * M1), 2049, 1.0, None) == SHAPE
    for rate in (NAN, INF):
        assert f(p(M1), p(2 * M1), p(3 * M1), 8, rate, None) == SHAPE
    for bad in (M1, M1 + 28, 2 * M1 + 4):
        assert f(p(M1), p(2 * M1), p(bad), 8, 1.0, None) == SHAPE
    for i in range(3):
        ptrs = [p(M1), p(2 * M1), p(3 * M1)]
        ptrs[i] = None
        assert f(*ptrs, 8, 1.0, None) == NULL
        ptrs[i] = p(5 * M1 + 2)
        assert f(*ptrs, 8, 1.0, None) == ALIGN


def _norm(L):
    a = L.MoeNormArgs()
    a.y, a.r, a.h, a.z, a.w_post, a.w_pre = (i * M1 for i in range(1, 7))
    a.q, a.q_scale = 7 * M1, 8 * M1
    a.M, a.H, a.post_norm, a.eps, a.residual_scale = 100, 256, 1, 1e-6, 1.0
    a.ldy = a.ldr = a.ldh = a.ldz = a.ldgate = 256
    return a


def test_norm_residual_refusals(L):
    f, a = L.load().moe_norm_residual, _norm(L)
    assert f(None, None) == NULL
    for bad in ({"dtype": 3}, {"stream_dtype": 1}, {"weight_dtype": 1}, {"dtype": 2}, {"stream_dtype": 7}):
        _refused(f, a, DTYPE, **bad)
    for bad in ({"M": -1}, {"M": 1 << 31}, {"H": 0}, {"H": 4}, {"H": 252}, {"H": 16392, "ldy": 16392}, {"ldy": 248}, {"ldy": 260}, {"ldr": 0},
                {"ldh": 257}, {"ldz": 128}, {"ldy": (1 << 40) + 8}, {"gate_mode": 4}, {"gate_mode": -1}, {"eps": -1e-6}, {"eps": NAN}, {"eps": INF},
                {"residual_scale": NAN}, {"residual_scale": INF}, {"weight_offset": NAN}, {"scale_mode": 2}, {"H": 248},
                {"gate_mode": 3, "gate": 9 * M1, "ldgate": 252},
                {"h": M1}, {"h": 2 * M1 + 16}, {"h": 2 * M1, "ldh": 264}, {"z": 2 * M1}, {"z": M1 + 512}, {"z": 3 * M1}, {"q": 4 * M1 + 64},
                {"q_scale": 7 * M1}, {"h": 5 * M1}, {"z": 6 * M1}, {"gate_mode": 1, "gate": 3 * M1}, {"gate_mode": 2, "gate": 4 * M1},
                {"gate_mode": 3, "gate": 7 * M1}, {"num_rows": 3 * M1}):
        _refused(f, a, SHAPE, **bad)
    for bad in ({"y": None}, {"h": None, "z": None, "q": None, "q_scale": None}, {"q": None}, {"q_scale": None}, {"gate_mode": 1}, {"gate_mode": 3}):
        _refused(f, a, NULL, **bad)
    for name in ("y", "r", "h", "z", "w_post", "w_pre", "q"):
        _refused(f, a, ALIGN, **{name: 9 * M1 + 8})
    for bad in ({"gate_mode": 1, "gate": 9 * M1 + 8}, {"gate_mode": 2, "gate": 9 * M1 + 2}, {"q_scale": 9 * M1 + 2}, {"num_rows": 9 * M1 + 1}):
        _refused(f, a, ALIGN, **bad)
    _refused(f, a, OK, M=0, y=None)


def _norm_grad(L):
    a = L.MoeNormBackwardArgs()
    for i, name in enumerate(("y", "h", "w_post", "w_pre", "dh", "dz", "dy", "dr", "dw_post", "dw_pre", "gate", "dgate", "workspace")):
        setattr(a, name, (i + 1) * M1)
    a.M, a.H, a.post_norm, a.eps, a.residual_scale, a.gate_mode = 100, 256, 1, 1e-6, 1.0, 1
    a.ldy = a.ldh = a.ldgate = a.lddh = a.lddz = a.lddy = a.lddr = a.lddgate = 256
    a.workspace_bytes = L.moe_norm_residual_workspace_size(100, 256)
    return a


def test_norm_residual_backward_refusals(L):
    f, a = L.load().moe_norm_residual_backward, _norm_grad(L)
    assert f(None, None) == NULL
    for bad in ({"dtype": 3}, {"stream_dtype": 1}, {"weight_dtype": 1}):
        _refused(f, a, DTYPE, **bad)
    for bad in ({"M": -1}, {"H": 12}, {"H": 16392}, {"ldy": 248}, {"ldh": 260}, {"lddh": 248}, {"lddz": 1}, {"lddy": 260}, {"lddr": 255},
                {"gate_mode": 3, "lddgate": 260}, {"gate_mode": 3, "ldgate": 248}, {"gate_mode": 0}, {"post_norm": 0}, {"eps": -1.0}, {"h": None},
                {"dy": 5 * M1}, {"dy": 6 * M1 + 16}, {"dy": 6 * M1, "lddy": 264}, {"dr": M1}, {"dr": 6 * M1}, {"dr": 5 * M1, "lddr": 264},
                {"dr": 7 * M1}, {"dw_pre": 9 * M1}, {"dw_post": 3 * M1}, {"dgate": 11 * M1}, {"dgate": 10 * M1 + 512}, {"workspace": M1},
                {"workspace": 9 * M1}, {"num_rows": 7 * M1}):
        _refused(f, a, SHAPE, **bad)
    for bad in ({"y": None}, {"dh": None, "dz": None}, {"dz": None}, {"gate": None}, {"workspace": None}):
        _refused(f, a, NULL, **bad)
    _refused(f, a, CAPACITY, workspace_bytes=a.workspace_bytes - 1)
    for name in ("y", "h", "w_post", "w_pre", "dh", "dz", "dy", "dr", "dw_post", "dw_pre", "gate", "dgate", "workspace"):
        _refused(f, a, ALIGN, **{name: 20 * M1 + 8})
    _refused(f, a, OK, M=0, dw_post=None, dw_pre=None, dgate=None)
    for M, H in ((-1, 256), (10, 0), (10, 12), (10, 16392), (1 << 31, 256)):
        assert L.moe_norm_residual_workspace_size(M, H) == 0
    assert 0 < L.moe_norm_residual_workspace_size(0, 8) <= L.moe_norm_residual_workspace_size(1 << 20, 16384) < 1 << 28


def test_records_have_the_headers_layout(L, tmp_path):
    """Sizes and the last field's offset of each record as the C compiler lays it out."""
    names = {"moe_route_scores_args": L.MoeRouteScoresArgs, "moe_route_scores_backward_args": L.MoeRouteScoresBackwardArgs,
             "moe_norm_args": L.MoeNormArgs, "moe_norm_backward_args": L.MoeNormBackwardArgs}
    lines = []
    for c, py in names.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{n} %zu\\n", offsetof({c}, {n}));' for n, _ in py._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "moe_block.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "t")], check=True)
    said = dict(line.split() for line in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, py in names.items():
        assert int(said[c]) == ctypes.sizeof(py)
        for n, _ in py._fields_:
            assert int(said[f"{c}.{n}"]) == getattr(py, n).offset
    header = open(os.path.join(ROOT, "include", "moe_block.h")).read()
    for name, value in (("MOE_SCORE_SOFTMAX", L.SCORE_SOFTMAX), ("MOE_SCORE_SIGMOID", L.SCORE_SIGMOID), ("MOE_GROUP_MAX", L.GROUP_MAX),
                        ("MOE_GROUP_TOP2", L.GROUP_TOP2), ("MOE_GATE_NONE", L.GATE_NONE), ("MOE_GATE_CHANNEL", L.GATE_CHANNEL),
                        ("MOE_GATE_TOKEN", L.GATE_TOKEN), ("MOE_GATE_FULL", L.GATE_FULL)):
        assert re.search(rf"#define {name}\s+{value}\b", header)


def test_binding_refusals(L):
    """Tensors of other shapes, types or layouts than the record can say."""
    l, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    L.make_route_scores_args(l, ids, w, bias=torch.zeros(8))
    for bad in ({"logits": l.double()}, {"logits": l[0]}, {"logits": l.t()}, {"topk_ids": ids.short()}, {"topk_ids": ids[:3]},
                {"topk_ids": ids.view(2, 4)}, {"topk_weights": w.half()}, {"topk_weights": w[:, :1]}, {"bias": torch.zeros(7)},
                {"bias": torch.zeros(8).half()}, {"bias": torch.zeros(16)[::2]}, {"num_tokens": torch.zeros(1)}):
        with pytest.raises(ValueError):
            L.make_route_scores_args(**{"logits": l, "topk_ids": ids, "topk_weights": w, **bad})
    for bad in ({"dlogits": l.half()}, {"dlogits": torch.zeros(4, 9)}, {"dweights": w[:3]}):
        with pytest.raises(ValueError):
            L.make_route_scores_backward_args(**{"logits": l, "topk_ids": ids, "dweights": w, "dlogits": l, **bad})
    with pytest.raises(ValueError):
        L.moe_route_balance(torch.zeros(7, dtype=torch.int32), torch.zeros(8), 1.0)
    with pytest.raises(ValueError):
        L.moe_route_balance(torch.zeros(8), torch.zeros(8), 1.0)

    y, wide, weight = torch.zeros(4, 256).bfloat16(), torch.zeros(4, 256), torch.zeros(256)
    args = L.make_norm_residual_args(y, h=wide, r=wide, w_post=weight, gate=weight)
    assert (args.gate_mode, args.post_norm, args.stream_dtype, args.weight_dtype) == (L.GATE_CHANNEL, 1, 2, 2)
    assert L.make_norm_residual_args(y, z=y, gate=torch.zeros(4, 1)).gate_mode == L.GATE_TOKEN
    assert L.make_norm_residual_args(y, z=y, gate=y).gate_mode == L.GATE_FULL
    for bad in ({"h": wide.half()}, {"h": wide, "r": y}, {"z": wide}, {"z": y[:3]}, {"h": wide[:, :128]}, {"w_post": weight[:255]},
                {"w_post": weight.half()}, {"w_post": weight, "w_pre": weight.bfloat16()}, {"w_post": weight, "post_norm": False},
                {"gate": torch.zeros(4)}, {"gate": wide}, {"gate": torch.zeros(4, 1).bfloat16()}, {"gate": torch.zeros(4, 2)[:, :1]},
                {"gate": weight.half()}, {"q": torch.zeros(4, 256, dtype=torch.uint8)}, {"q_scale": torch.zeros(4, 2)},
                {"q": torch.zeros(4, 256), "q_scale": torch.zeros(4, 2)}, {"q": torch.zeros(4, 256, dtype=torch.uint8), "q_scale": torch.zeros(4, 3)},
                {"num_rows": torch.zeros(1)}, {"z": y.t()}):
        with pytest.raises(ValueError):
            L.make_norm_residual_args(y, **bad)
    for bad in ({"dgate": weight}, {"gate": weight, "dgate": weight.bfloat16()}, {"gate": torch.zeros(4, 1), "dgate": torch.zeros(4)},
                {"gate": y, "dgate": wide}, {"dz": wide}, {"dh": wide, "dr": y}, {"dw_pre": weight[:8]}, {"dw_post": weight.bfloat16()}):
        with pytest.raises(ValueError):
            L.make_norm_residual_backward_args(y, **bad)
