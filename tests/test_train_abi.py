"""Host-side argument checks of the training entry points (no GPU needed)."""

import ctypes

import pytest

NULL, SHAPE, ALIGN, CAPACITY, DTYPE, OK = 1, 2, 3, 4, 5, 0


@pytest.fixture(scope="module")
def L():
    from fp8_block_scale_gb300 import _lib
    from fp8_block_scale_gb300.build import build
    build()
    _lib.load()
    return _lib


def _grouped(L):
    a = L.MoeGroupedArgs()
    a.x, a.w, a.y, a.group_start, a.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    a.rows, a.E, a.N, a.K, a.ldx, a.ldy = 100, 4, 64, 32, 32, 64
    return a


def _refused(fn, args, want, **fields):
    old = {k: getattr(args, k) for k in fields}
    for k, v in fields.items():
        setattr(args, k, v)
    got = fn(ctypes.byref(args), None)
    for k, v in old.items():
        setattr(args, k, v)
    assert got == want, (fields, got)


def test_grouped_gemm_refusals(L):
    f = L.load().moe_grouped_gemm
    a = _grouped(L)
    assert f(None, None) == NULL
    for bad in (2, -1, 7):
        _refused(f, a, DTYPE, dtype=bad)
    for bad in ({"E": 0}, {"E": 2049}, {"N": 0}, {"N": 60}, {"K": 36, "ldx": 40}, {"rows": -1}, {"rows": 1 << 31},
                {"ldx": 24}, {"ldx": 36}, {"ldy": 56}, {"ldy": 68}, {"direction": 2}, {"epilogue": 2},
                {"epilogue": 1, "direction": 1}, {"epilogue": 1, "N": 72, "ldy": 40}, {"R": -1},
                {"direction": 1},                                         # x is N wide then, ldx = 32 < 64
                {"epilogue": 1, "pre": 16 << 20, "ldpre": 56},
                {"y": 1 << 20}, {"y": (1 << 20) + 3200}, {"y": 2 << 20},   # overlaps of the output
                {"epilogue": 1, "pre": 4 << 20, "ldpre": 64}):
        _refused(f, a, SHAPE, **bad)
    for name in ("x", "w", "y", "group_start", "group_rows"):
        _refused(f, a, NULL, **{name: None})
    for name in ("x", "w", "y"):
        _refused(f, a, ALIGN, **{name: (32 << 20) + 8})
    _refused(f, a, OK, rows=0)


def test_grouped_wgrad_refusals(L):
    f = L.load().moe_grouped_wgrad
    a = L.MoeGroupedWgradArgs()
    a.dy, a.x, a.dw, a.group_start, a.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    a.rows, a.E, a.N, a.K, a.lddy, a.ldx = 100, 4, 64, 32, 64, 32
    assert f(None, None) == NULL
    for bad in ({"dtype": 2}, {"dw_dtype": 1}, {"dw_dtype": 3}, {"accumulate": 1}):
        _refused(f, a, DTYPE, **bad)
    for bad in ({"E": 0}, {"N": 12}, {"K": 20}, {"rows": -1}, {"lddy": 56}, {"ldx": 36}, {"dw": 1 << 20}, {"dw": 2 << 20}):
        _refused(f, a, SHAPE, **bad)
    for name in ("dy", "x", "dw", "group_start", "group_rows"):
        _refused(f, a, NULL, **{name: None})
    for name in ("dy", "x", "dw"):
        _refused(f, a, ALIGN, **{name: (32 << 20) + 4})


def test_swiglu_backward_refusals(L):
    f = L.load().moe_swiglu_backward
    a = L.MoeSwigluBackwardArgs()
    a.dh, a.pre, a.dpre, a.h = 1 << 20, 2 << 20, 4 << 20, 8 << 20
    a.rows, a.I, a.lddh, a.ldpre, a.lddpre, a.ldh, a.R = 100, 64, 64, 128, 128, 64, 100
    assert f(None, None) == NULL
    _refused(f, a, DTYPE, dtype=2)
    for bad in ({"I": 4}, {"I": 20}, {"rows": -1}, {"lddh": 56}, {"ldpre": 120}, {"lddpre": 132}, {"ldh": 60}, {"R": -1},
                {"dpre": (2 << 20) + 256}, {"dpre": 1 << 20}, {"h": 2 << 20}, {"h": 4 << 20}, {"h": (1 << 20) + 128},
                {"dpre": 2 << 20, "lddpre": 136}):                       # in place only at the same stride
        _refused(f, a, SHAPE, **bad)
    for name in ("dh", "pre", "dpre"):
        _refused(f, a, NULL, **{name: None})
        _refused(f, a, ALIGN, **{name: (32 << 20) + 8})
    _refused(f, a, OK, rows=0)


def test_rows_and_groups_refusals(L):
    lib = L.load()
    p = ctypes.c_void_p
    gather = [p(1 << 20), 10, 64, 64, p(2 << 20), 20, 64, p(3 << 20), 2, None, 0, None]

    def g(want, **at):
        args = list(gather)
        for k, v in at.items():
            args[int(k[1:])] = v
        assert lib.moe_gather_rows(*args) == want, at

    g(DTYPE, a10=3)
    g(SHAPE, a1=-1), g(SHAPE, a2=4), g(SHAPE, a2=12), g(SHAPE, a3=56), g(SHAPE, a6=68), g(SHAPE, a8=0), g(SHAPE, a1=1 << 31)
    g(SHAPE, a4=p((1 << 20) + 1024))
    g(NULL, a0=None), g(NULL, a4=None), g(NULL, a7=None)
    g(ALIGN, a0=p((1 << 20) + 8)), g(ALIGN, a4=p((4 << 20) + 4))
    g(OK, a5=0)
    total = [p(1 << 20), 20, 64, 64, p(2 << 20), 10, 64, p(3 << 20), 2, 0, 0, None]

    def s(want, **at):
        args = list(total)
        for k, v in at.items():
            args[int(k[1:])] = v
        assert lib.moe_sum_routes(*args) == want, at

    s(DTYPE, a10=-1)
    s(SHAPE, a1=-1), s(SHAPE, a2=0), s(SHAPE, a3=63), s(SHAPE, a6=32), s(SHAPE, a8=0), s(SHAPE, a4=p(1 << 20))
    s(NULL, a0=None), s(NULL, a4=None), s(NULL, a7=None), s(ALIGN, a4=p((2 << 20) + 2)), s(OK, a5=0)
    groups = [p(4096), 640, p(8192), 10, p(64), 64, 32, 8, p(128), p(256), None, None]

    def pg(want, **at):
        args = list(groups)
        for k, v in at.items():
            args[int(k[1:])] = v
        assert lib.moe_plan_groups(*args) == want, at

    pg(SHAPE, a5=12), pg(SHAPE, a7=0), pg(SHAPE, a7=2049), pg(SHAPE, a6=-1), pg(SHAPE, a3=-1)
    pg(CAPACITY, a1=639)
    for k in (0, 2, 4, 8, 9):
        pg(NULL, **{f"a{k}": None})


def test_adamw_refusals(L):
    lib = L.load()
    assert lib.moe_adamw_table_bytes(0) == 0 and lib.moe_adamw_table_bytes(65537) == 0
    size = lib.moe_adamw_table_bytes(1)
    t = (L.MoeAdamWTensor * 1)()
    e = t[0]
    e.param, e.grad, e.exp_avg, e.exp_avg_sq, e.n, e.grad_dtype = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 100, 2
    chunks, types = ctypes.c_int64(), ctypes.c_int32()
    table = ctypes.c_void_p(8 << 20)

    def init(want, bits=32, count=1, tab=table, nbytes=size, **fields):
        old = {k: getattr(e, k) for k in fields}
        for k, v in fields.items():
            setattr(e, k, v)
        got = lib.moe_adamw_table_init(t, count, bits, tab, nbytes, ctypes.byref(chunks), ctypes.byref(types), None)
        for k, v in old.items():
            setattr(e, k, v)
        assert got == want, (fields, got)

    init(DTYPE, bits=16), init(SHAPE, count=0), init(NULL, tab=None), init(CAPACITY, nbytes=size - 1)
    init(ALIGN, tab=ctypes.c_void_p((8 << 20) + 8))
    init(SHAPE, n=-1), init(SHAPE, weight_decay=float("nan")), init(DTYPE, grad_dtype=3), init(DTYPE, model=5 << 20, model_dtype=2)
    for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
        init(NULL, **{name: None}), init(ALIGN, **{name: (1 << 20) + 4})
    init(NULL, bits=8)
    init(ALIGN, bits=8, exp_avg_scale=4098, exp_avg_sq_scale=4096)

    a = L.MoeAdamWArgs()
    a.table, a.chunks, a.count, a.state_bits, a.step = 1 << 20, 1, 1, 32, 1
    a.lr, a.beta1, a.beta2, a.eps = 1e-3, 0.9, 0.99, 1e-8
    f = lib.moe_adamw_step
    assert f(None, None) == NULL
    _refused(f, a, DTYPE, state_bits=4)
    nan = float("nan")
    for bad in ({"count": 0}, {"chunks": -1}, {"grad_types": 8}, {"grad_types": -1}, {"step": 0}, {"lr": -1.0}, {"lr": nan}, {"lr": float("inf")}, {"eps": -1.0},
                {"beta1": 1.0}, {"beta1": nan}, {"beta2": -0.1}):
        _refused(f, a, SHAPE, **bad)
    _refused(f, a, NULL, table=None)
    _refused(f, a, OK, chunks=0)


def test_python_wrappers_refuse_what_the_records_cannot_say(L):
    import torch
    bf = torch.bfloat16
    x, w, y = torch.zeros(6, 32, dtype=bf), torch.zeros(2, 64, 32, dtype=bf), torch.zeros(6, 64, dtype=bf)
    s = torch.zeros(2, dtype=torch.int32)
    L.make_grouped_args(x, w, y, s, s)
    with pytest.raises(ValueError):
        L.make_grouped_args(x.t().contiguous().t(), w, y, s, s)           # rows not contiguous
    with pytest.raises(ValueError):
        L.make_grouped_args(x, w.transpose(1, 2), y, s, s)
    with pytest.raises(ValueError):
        L.make_grouped_args(x, w, y[:, :32], s, s)
    with pytest.raises(ValueError):
        L.make_grouped_args(x, w, y, s[:1], s)
    with pytest.raises(ValueError):
        L.make_grouped_args(x, w, y, s.long(), s)
    with pytest.raises(ValueError):
        L.make_grouped_args(x.half(), w, y, s, s)
    with pytest.raises(ValueError):
        L.make_grouped_wgrad_args(y, x, torch.zeros(2, 32, 64, dtype=bf), s, s)
    with pytest.raises(ValueError):
        L.make_swiglu_backward_args(x, y[:, :32], y)
    with pytest.raises(ValueError):
        L.AdamWTable([])
