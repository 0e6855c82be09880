"""Host side of the training operators and of the expert layer (no GPU needed)."""

import pytest
import torch

from fp8_block_scale_gb300.training import ExpertLayer


@pytest.fixture(scope="module")
def L():
    from fp8_block_scale_gb300 import _lib
    from fp8_block_scale_gb300.build import build
    build()
    _lib.load()
    return _lib


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_only_bf16_weights_are_quantised(L, dtype):
    """The kernel reads BF16 bits: another type would give wrong codes."""
    w = torch.zeros(2, 128, 128, dtype=dtype)
    q, s = torch.zeros(2, 128, 128, dtype=torch.uint8), torch.zeros(2, 1, 1)
    with pytest.raises(ValueError):
        L.moe_quantize_weight_128x128(w, q, s)
    layer = object.__new__(ExpertLayer)
    layer.models = [w, w]
    with pytest.raises(ValueError):
        layer.quantized()


@pytest.fixture
def layer(monkeypatch):
    """A layer of 8 tokens, H 64, E 4 without its buffers; library calls fail the test."""
    from fp8_block_scale_gb300 import training

    class NoCalls:
        def __getattr__(self, name):
            pytest.fail(f"{name} was reached")

    monkeypatch.setattr(training, "L", NoCalls())
    layer = object.__new__(ExpertLayer)
    layer.M, layer.H, layer.I, layer.E, layer.top_k, layer.dtype = 8, 64, 16, 4, 2, torch.bfloat16
    return layer


@pytest.mark.parametrize("logits", [
    torch.zeros(9, 4), torch.zeros(7, 4), torch.zeros(8, 5), torch.zeros(8), torch.zeros(8, 4, dtype=torch.float16),
    torch.zeros(4, 8).t(), torch.zeros(8, 8)[:, ::2]])
def test_layer_refuses_logits_that_its_buffers_do_not_hold(layer, logits):
    """More rows would be written past the ids and weights; fewer would leave those of a step before."""
    with pytest.raises(ValueError):
        layer.route(logits)


@pytest.mark.parametrize("x", [torch.zeros(n, w, dtype=d) for n, w, d in (
    (9, 64, torch.bfloat16), (7, 64, torch.bfloat16), (8, 72, torch.bfloat16), (8, 64, torch.float16))])
def test_layer_refuses_other_rows(layer, x):
    with pytest.raises(ValueError):
        layer.forward(x)
    with pytest.raises(ValueError):
        layer.backward(x)


def test_argument_records_keep_their_tensors(L):
    """A temporary that only the record knows must live as long as the record."""
    import gc
    import weakref

    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = torch.zeros
    records = [
        (lambda *t: L.make_grouped_args(*t[:5], epilogue=L.GROUPED_SWIGLU, pre=t[5], route_ids=t[6], route_weights=t[7],
                                        device_status=t[8]),
         [z(6, 32, dtype=bf), z(2, 64, 32, dtype=bf), z(6, 32, dtype=bf), z(2, dtype=i32), z(2, dtype=i32), z(6, 64, dtype=bf),
          z(6, dtype=i32), z(9, dtype=f32), z(1, dtype=i32)]),
        (lambda *t: L.make_grouped_wgrad_args(*t[:5], device_status=t[5]),
         [z(6, 64, dtype=bf), z(6, 32, dtype=bf), z(2, 64, 32), z(2, dtype=i32), z(2, dtype=i32), z(1, dtype=i32)]),
        (lambda *t: L.make_swiglu_backward_args(*t[:3], h=t[3], route_ids=t[4], num_rows=t[5], route_weights=t[6], dweights=t[7]),
         [z(6, 32, dtype=bf), z(6, 64, dtype=bf), z(6, 64, dtype=bf), z(6, 32, dtype=bf), z(6, dtype=i32), z(1, dtype=i32), z(9), z(9)]),
    ]
    while records:
        make, tensors = records.pop()
        args = make(*tensors)
        refs = [weakref.ref(t) for t in tensors]
        del tensors
        gc.collect()
        assert all(r() is not None for r in refs)
        del args
        gc.collect()
        assert all(r() is None for r in refs)


def test_current_stream_without_torchs_raw_lookups(L, monkeypatch):
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        with monkeypatch.context() as m:
            m.delattr(torch._C, name, raising=False)
            assert L._stream().value == 0x1234
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x100 + d, raising=False)
    assert L._stream().value == 0x103
    assert L._stream(Stream).value == 0x1234


def test_a_single_row_may_have_any_stride(L):
    """torch calls a transposed column [1, n] contiguous with a row stride of 1."""
    bf = torch.bfloat16
    one = torch.zeros(32, 1, dtype=bf).t()
    assert one.shape == (1, 32) and one.stride() == (1, 1) and one.is_contiguous()
    w, y, s = torch.zeros(2, 64, 32, dtype=bf), torch.zeros(64, 1, dtype=bf).t(), torch.zeros(2, dtype=torch.int32)
    args = L.make_grouped_args(one, w, y, s, s)
    assert (args.ldx, args.ldy) == (32, 64)
    args = L.make_grouped_wgrad_args(y, one, torch.zeros_like(w), s, s)
    assert (args.lddy, args.ldx) == (64, 32)
    args = L.make_swiglu_backward_args(one, y, torch.zeros(1, 64, dtype=bf), h=torch.zeros(32, 1, dtype=bf).t())
    assert (args.lddh, args.ldpre, args.lddpre, args.ldh) == (32, 64, 64, 32)
    with pytest.raises(ValueError):
        L.make_grouped_args(torch.zeros(32, 2, dtype=bf).t(), w, torch.zeros(2, 64, dtype=bf), s, s)


def test_columns_beside_one_another_do_not_overlap(L):
    """Outputs and inputs may be columns of one wider buffer; columns that share an element may not."""
    SHAPE, bf, i32 = 2, torch.bfloat16, torch.int32
    lib = L.load()
    buf, s = torch.zeros(20, 256, dtype=bf), torch.zeros(2, dtype=i32)
    cols = lambda a, n: buf[:, a:a + n]                                              # noqa: E731
    w = torch.zeros(2, 64, 32, dtype=bf)

    def status(make, call, *a, **kw):
        args = make(*a, **kw)
        return getattr(lib, call)(args, None)

    def gemm(x, y, **kw):
        return status(L.make_grouped_args, "moe_grouped_gemm", x, w, y, s, s, **kw)

    def back(*a, **kw):
        return status(L.make_swiglu_backward_args, "moe_swiglu_backward", *a, **kw)

    # (without a device the calls end there; what counts is that their sizes are not refused)
    glu = dict(epilogue=L.GROUPED_SWIGLU)
    assert gemm(cols(0, 32), cols(32, 64)) != SHAPE and gemm(cols(0, 32), cols(24, 64)) == SHAPE
    assert gemm(cols(64, 32), cols(0, 64)) != SHAPE and gemm(cols(56, 32), cols(0, 64)) == SHAPE
    assert gemm(cols(128, 32), cols(160, 32), pre=cols(0, 64), **glu) != SHAPE
    assert gemm(cols(128, 32), cols(160, 32), pre=cols(104, 64), **glu) == SHAPE
    assert gemm(cols(128, 32), cols(160, 32), pre=cols(176, 64), **glu) == SHAPE
    # rows from one on: the end of a row and the start of the next are neighbours too
    assert gemm(buf.view(-1)[128:128 + 19 * 256].view(19, 256)[:, :32], buf[:19, 0:64]) != SHAPE
    assert gemm(buf.view(-1)[240:240 + 19 * 256].view(19, 256)[:, :32], buf[:19, 0:64]) == SHAPE
    # another stride cannot be told apart
    assert gemm(buf.view(40, 128)[:20, :32], cols(64, 64)) == SHAPE
    assert back(cols(0, 32), cols(32, 64), cols(96, 64), h=cols(160, 32)) != SHAPE
    assert back(cols(0, 32), cols(32, 64), cols(88, 64), h=cols(160, 32)) == SHAPE
    assert back(cols(0, 32), cols(32, 64), cols(96, 64), h=cols(152, 32)) == SHAPE
    assert back(cols(0, 32), cols(32, 64), cols(32, 64), h=cols(0, 32)) != SHAPE      # in place
    rows = lambda f, a, b: getattr(lib, f)(                                          # noqa: E731
        a.data_ptr(), 20, 64, 256, b.data_ptr(), 20, 256, s.data_ptr(), *((1, None) if "gather" in f else (1, 0)), 0, None)
    for f in ("moe_gather_rows", "moe_sum_routes"):
        assert rows(f, cols(0, 64), cols(64, 64)) != SHAPE and rows(f, cols(0, 64), cols(56, 64)) == SHAPE


def test_sizes_whose_products_pass_64_bits_are_refused(L):
    import ctypes

    SHAPE, p, lib = 2, ctypes.c_void_p, L.load()
    for M, k in ((1 << 33, 1 << 30), (1 << 34, 1 << 29), (1 << 32, 1), (1 << 40, 1 << 24), (1 << 62, 4)):
        assert lib.moe_gather_rows(p(1 << 20), M, 64, 64, p(2 << 20), 20, 64, p(3 << 20), k, None, 0, None) == SHAPE, (M, k)
        assert lib.moe_sum_routes(p(1 << 20), 20, 64, 64, p(2 << 20), M, 64, p(3 << 20), k, 0, 0, None) == SHAPE, (M, k)
    far = 1 << 62
    assert lib.moe_gather_rows(p(1 << 20), 5, 64, far, p(2 << 20), 20, 64, p(3 << 20), 1, None, 0, None) == SHAPE
    assert lib.moe_sum_routes(p(1 << 20), 20, 64, 64, p(2 << 20), 5, far, p(3 << 20), 1, 0, 0, None) == SHAPE
    a = L.MoeGroupedArgs()
    a.x, a.w, a.y, a.group_start, a.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    a.rows, a.E, a.N, a.K, a.ldx, a.ldy = 100, 4, 64, 32, far, 64
    assert lib.moe_grouped_gemm(ctypes.byref(a), None) == SHAPE
    a.ldx, a.E, a.N, a.K = 1 << 30, 2048, 1 << 30, 1 << 30
    a.ldy = 1 << 30
    assert lib.moe_grouped_gemm(ctypes.byref(a), None) == SHAPE
    b = L.MoeGroupedWgradArgs()
    b.dy, b.x, b.dw, b.group_start, b.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    b.rows, b.E, b.N, b.K, b.lddy, b.ldx = 100, 2048, 1 << 30, 1 << 30, 1 << 30, 1 << 30
    assert lib.moe_grouped_wgrad(ctypes.byref(b), None) == SHAPE
    c = L.MoeSwigluBackwardArgs()
    c.dh, c.pre, c.dpre, c.rows, c.I, c.lddh, c.ldpre, c.lddpre = 1 << 20, 2 << 20, 4 << 20, 100, 64, far, 128, 128
    assert lib.moe_swiglu_backward(ctypes.byref(c), None) == SHAPE


def test_misaligned_tables_are_refused(L):
    """A 4-byte element off its alignment would fault on the device."""
    import ctypes

    ALIGN, p, lib, odd = 3, ctypes.c_void_p, L.load(), (32 << 20) + 2

    def refused(call, args, *names):
        for name in names:
            old = getattr(args, name)
            setattr(args, name, odd)
            assert getattr(lib, call)(ctypes.byref(args), None) == ALIGN, (call, name)
            setattr(args, name, old)

    a = L.MoeGroupedArgs()
    a.x, a.w, a.y, a.group_start, a.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    a.rows, a.E, a.N, a.K, a.ldx, a.ldy, a.epilogue = 100, 4, 64, 32, 32, 64, 1
    refused("moe_grouped_gemm", a, "group_start", "group_rows", "route_ids", "route_weights", "device_status")
    b = L.MoeGroupedWgradArgs()
    b.dy, b.x, b.dw, b.group_start, b.group_rows = 1 << 20, 2 << 20, 4 << 20, 8 << 20, 9 << 20
    b.rows, b.E, b.N, b.K, b.lddy, b.ldx = 100, 4, 64, 32, 64, 32
    refused("moe_grouped_wgrad", b, "group_start", "group_rows", "device_status")
    c = L.MoeSwigluBackwardArgs()
    c.dh, c.pre, c.dpre, c.rows, c.I, c.lddh, c.ldpre, c.lddpre = 1 << 20, 2 << 20, 4 << 20, 100, 64, 64, 128, 128
    refused("moe_swiglu_backward", c, "route_ids", "num_rows", "route_weights", "dweights")
    d = L.MoeAdamWArgs()
    d.table, d.chunks, d.count, d.state_bits, d.step, d.lr = 1 << 20, 1, 1, 32, 1, 1e-3
    refused("moe_adamw_step", d, "table", "grad_scale", "skip")
    for k in (7, 9):
        v = [p(1 << 20), 10, 64, 64, p(2 << 20), 20, 64, p(3 << 20), 2, None, 0, None]
        v[k] = p(odd)
        assert lib.moe_gather_rows(*v) == ALIGN
    assert lib.moe_sum_routes(p(1 << 20), 20, 64, 64, p(2 << 20), 10, 64, p(odd), 2, 0, 0, None) == ALIGN
    for k in (0, 2, 4, 8, 9, 10):
        v = [p(4096), 640, p(8192), 10, p(64), 64, 32, 8, p(128), p(256), p(512), None]
        v[k] = p(odd)
        assert lib.moe_plan_groups(*v) == ALIGN, k


def test_plan_groups_takes_int32_plans_only(L):
    """64-bit ids would be read as pairs of 32-bit ones."""
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t)                             # noqa: E731
    for k in range(3):
        plan = [z(32), z(4), z(1)]
        plan[k] = z(plan[k].numel(), torch.int64)
        with pytest.raises(ValueError):
            L.moe_plan_groups(*plan, 8, 6, z(4), z(4))
    with pytest.raises(ValueError):
        L.moe_plan_groups(z(64)[::2], z(4), z(1), 8, 6, z(4), z(4))


@pytest.mark.parametrize("name", ["grouped.cu", "rows.cu", "adamw.cu"])
def test_training_kernels_have_bounds_checks(name):
    """What the bounds-checking build reports about a file is worth something only where it checks."""
    import os

    import fp8_block_scale_gb300
    with open(os.path.join(os.path.dirname(fp8_block_scale_gb300.__file__), "csrc", name)) as f:
        text = f.read()
    assert "MOE_BOUNDS_TU()" in text and text.count("MOE_IN_BOUNDS(") >= 4
