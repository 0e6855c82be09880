"""ctypes binding of libmoe_fp8.so (the C ABI declared in include/moe_fp8.h).

Argument marshalling only: every function forwards device pointers, sizes
and the current torch stream to the C entry point of the same name and raises
``MoeError`` on a non-zero status.  There is no fallback: if the shared
library is missing, loading fails loudly.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_fp8.so")
LIB_DEBUG_PATH = os.path.join(_PKG, "libmoe_fp8_debug.so")  # the bounds-checking build

MOE_OK = 0
STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN", 4: "MOE_ERR_CAPACITY",
    5: "MOE_ERR_DTYPE", 6: "MOE_ERR_DEVICE", 7: "MOE_ERR_CUDA", 8: "MOE_ERR_TIMEOUT",
}
MOE_DEV_TIMEOUT = 0x1
MOE_DEV_BAD_EXPERT = 0x2
MOE_DEV_BAD_SCALE = 0x4
MOE_DEV_BAD_GROUP = 0x8


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


class MoeFwdArgs(ctypes.Structure):
    """Mirror of ``struct moe_fwd_args``."""
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("a_scale", ctypes.c_void_p),
        ("w13", ctypes.c_void_p),
        ("w13_scale", ctypes.c_void_p),
        ("w2", ctypes.c_void_p),
        ("w2_scale", ctypes.c_void_p),
        ("topk_weights", ctypes.c_void_p),
        ("sorted_token_ids", ctypes.c_void_p),
        ("expert_ids", ctypes.c_void_p),
        ("num_tokens_post_padded", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p),
        ("debug_q_inter", ctypes.c_void_p),
        ("debug_s_inter", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("sorted_cap", ctypes.c_int64),
        ("blocks_cap", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_size_t),
        ("H", ctypes.c_int32),
        ("I", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("block_m", ctypes.c_int32),
        ("routed_scale", ctypes.c_float),
        ("profile_events", ctypes.POINTER(ctypes.c_void_p)),
        ("tile_mode", ctypes.c_int32),
        ("scale_mode", ctypes.c_int32),
    ]


TILE_AUTO, TILE_SINGLE, TILE_PAIR, TILE_VECTOR = 0, 1, 2, 3
W4A8_AUTO, W4A8_CUDA_CORES = 0, 1
SCALES_FP32, SCALES_UE8M0 = 0, 1


class MoeW4A8Args(ctypes.Structure):
    """Mirror of ``struct moe_w4a8_args`` (include/moe_w4a8.h)."""
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("a_scale", ctypes.c_void_p),
        ("w13", ctypes.c_void_p),
        ("w13_scale", ctypes.c_void_p),
        ("w2", ctypes.c_void_p),
        ("w2_scale", ctypes.c_void_p),
        ("topk_weights", ctypes.c_void_p),
        ("sorted_token_ids", ctypes.c_void_p),
        ("expert_ids", ctypes.c_void_p),
        ("num_tokens_post_padded", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p),
        ("debug_q_inter", ctypes.c_void_p),
        ("debug_s_inter", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("sorted_cap", ctypes.c_int64),
        ("blocks_cap", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_size_t),
        ("H", ctypes.c_int32),
        ("I", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("block_m", ctypes.c_int32),
        ("routed_scale", ctypes.c_float),
        ("path", ctypes.c_int32),
    ]


GROUPED_FORWARD, GROUPED_INPUT_GRADIENT = 0, 1
GROUPED_PLAIN, GROUPED_SWIGLU = 0, 1
TYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class MoeGroupedArgs(ctypes.Structure):
    """Mirror of ``struct moe_grouped_args`` (include/moe_train.h)."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("pre", ctypes.c_void_p),
        ("group_start", ctypes.c_void_p),
        ("group_rows", ctypes.c_void_p),
        ("route_ids", ctypes.c_void_p),
        ("route_weights", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("ldx", ctypes.c_int64),
        ("ldy", ctypes.c_int64),
        ("ldpre", ctypes.c_int64),
        ("R", ctypes.c_int64),
        ("E", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("direction", ctypes.c_int32),
        ("epilogue", ctypes.c_int32),
    ]


class MoeGroupedWgradArgs(ctypes.Structure):
    """Mirror of ``struct moe_grouped_wgrad_args``."""
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("dw", ctypes.c_void_p),
        ("group_start", ctypes.c_void_p),
        ("group_rows", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("lddy", ctypes.c_int64),
        ("ldx", ctypes.c_int64),
        ("E", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("dw_dtype", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
    ]


class MoeSwigluBackwardArgs(ctypes.Structure):
    """Mirror of ``struct moe_swiglu_backward_args``."""
    _fields_ = [
        ("dh", ctypes.c_void_p),
        ("pre", ctypes.c_void_p),
        ("dpre", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("route_ids", ctypes.c_void_p),
        ("num_rows", ctypes.c_void_p),
        ("route_weights", ctypes.c_void_p),
        ("dweights", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("lddh", ctypes.c_int64),
        ("ldpre", ctypes.c_int64),
        ("lddpre", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("R", ctypes.c_int64),
        ("I", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class MoeAdamWTensor(ctypes.Structure):
    """Mirror of ``struct moe_adamw_tensor``."""
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("model", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("exp_avg_scale", ctypes.c_void_p),
        ("exp_avg_sq_scale", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("weight_decay", ctypes.c_double),
        ("grad_dtype", ctypes.c_int32),
        ("model_dtype", ctypes.c_int32),
    ]


class MoeAdamWArgs(ctypes.Structure):
    """Mirror of ``struct moe_adamw_args``."""
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("grad_scale", ctypes.c_void_p),
        ("skip", ctypes.c_void_p),
        ("chunks", ctypes.c_int64),
        ("step", ctypes.c_int64),
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("seed", ctypes.c_uint32),
        ("count", ctypes.c_int32),
        ("state_bits", ctypes.c_int32),
        ("grad_types", ctypes.c_int32),
    ]


SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


class MoeRouteScoresArgs(ctypes.Structure):
    """Mirror of ``struct moe_route_scores_args`` (include/moe_block.h)."""
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("topk_ids", ctypes.c_void_p),
        ("topk_weights", ctypes.c_void_p),
        ("num_tokens", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("ldlogits", ctypes.c_int64),
        ("E", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("id_bits", ctypes.c_int32),
        ("routed_scale", ctypes.c_float),
    ]


class MoeRouteScoresBackwardArgs(ctypes.Structure):
    """Mirror of ``struct moe_route_scores_backward_args``."""
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("topk_ids", ctypes.c_void_p),
        ("dweights", ctypes.c_void_p),
        ("dlogits", ctypes.c_void_p),
        ("num_tokens", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("ldlogits", ctypes.c_int64),
        ("lddlogits", ctypes.c_int64),
        ("E", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("id_bits", ctypes.c_int32),
        ("routed_scale", ctypes.c_float),
    ]


class MoeNormArgs(ctypes.Structure):
    """Mirror of ``struct moe_norm_args``."""
    _fields_ = [
        ("y", ctypes.c_void_p),
        ("r", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("w_post", ctypes.c_void_p),
        ("w_pre", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("q_scale", ctypes.c_void_p),
        ("num_rows", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("ldy", ctypes.c_int64),
        ("ldr", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("ldz", ctypes.c_int64),
        ("ldgate", ctypes.c_int64),
        ("H", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("stream_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32),
        ("post_norm", ctypes.c_int32),
        ("scale_mode", ctypes.c_int32),
        ("residual_scale", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("eps", ctypes.c_float),
    ]


class MoeNormBackwardArgs(ctypes.Structure):
    """Mirror of ``struct moe_norm_backward_args``."""
    _fields_ = [
        ("y", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("w_post", ctypes.c_void_p),
        ("w_pre", ctypes.c_void_p),
        ("dh", ctypes.c_void_p),
        ("dz", ctypes.c_void_p),
        ("dy", ctypes.c_void_p),
        ("dr", ctypes.c_void_p),
        ("dgate", ctypes.c_void_p),
        ("dw_post", ctypes.c_void_p),
        ("dw_pre", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("num_rows", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("M", ctypes.c_int64),
        ("ldy", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("ldgate", ctypes.c_int64),
        ("lddh", ctypes.c_int64),
        ("lddz", ctypes.c_int64),
        ("lddy", ctypes.c_int64),
        ("lddr", ctypes.c_int64),
        ("lddgate", ctypes.c_int64),
        ("H", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("stream_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32),
        ("post_norm", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
        ("residual_scale", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("eps", ctypes.c_float),
    ]


_libs = {}
_active = LIB_PATH

_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_plan_capacity": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]),
    "moe_plan_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "moe_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_prep_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_void_p]),
    "moe_requant_scales_ue8m0": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                                ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "moe_route_topk": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "moe_route_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "moe_quantize_act_1x128": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p]),
    "moe_quantize_act_1x128_ue8m0": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                                    ctypes.c_void_p, ctypes.c_void_p]),
    "moe_quantize_weight_128x128": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_forward_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_int, ctypes.c_int, ctypes.c_int64]),
    "moe_workspace_init": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_fp8_block_scale_forward": (ctypes.c_int, [ctypes.POINTER(MoeFwdArgs), ctypes.c_void_p]),
    "moe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_void_p]),
    "moe_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "moe_fp8_block_scale_forward_noalloc": (ctypes.c_int, [ctypes.POINTER(MoeFwdArgs), ctypes.c_void_p]),
    "moe_quantize_act_per_row": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p]),
    "moe_quantize_weight_k32": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p]),
    "moe_w4a8_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "moe_w4a8_forward": (ctypes.c_int, [ctypes.POINTER(MoeW4A8Args), ctypes.c_void_p]),
    "moe_plan_groups": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_gather_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_int, ctypes.c_void_p]),
    "moe_sum_routes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_void_p]),
    "moe_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(MoeGroupedArgs), ctypes.c_void_p]),
    "moe_grouped_wgrad": (ctypes.c_int, [ctypes.POINTER(MoeGroupedWgradArgs), ctypes.c_void_p]),
    "moe_swiglu_backward": (ctypes.c_int, [ctypes.POINTER(MoeSwigluBackwardArgs), ctypes.c_void_p]),
    "moe_adamw_table_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "moe_adamw_table_init": (ctypes.c_int, [ctypes.POINTER(MoeAdamWTensor), ctypes.c_int, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64),
                                            ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p]),
    "moe_adamw_step": (ctypes.c_int, [ctypes.POINTER(MoeAdamWArgs), ctypes.c_void_p]),
    "moe_route_scores": (ctypes.c_int, [ctypes.POINTER(MoeRouteScoresArgs), ctypes.c_void_p]),
    "moe_route_scores_backward": (ctypes.c_int, [ctypes.POINTER(MoeRouteScoresBackwardArgs), ctypes.c_void_p]),
    "moe_route_balance": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_float, ctypes.c_void_p]),
    "moe_norm_residual": (ctypes.c_int, [ctypes.POINTER(MoeNormArgs), ctypes.c_void_p]),
    "moe_norm_residual_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "moe_norm_residual_backward": (ctypes.c_int, [ctypes.POINTER(MoeNormBackwardArgs), ctypes.c_void_p]),
    "moe_debug_bounds_enabled": (ctypes.c_int, []),
    "moe_debug_bounds_selftest": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                                 ctypes.c_void_p]),
    "moe_debug_bounds_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_char_p),
                                             ctypes.POINTER(ctypes.c_int32), ctypes.c_int]),
}


def load(path=None):
    """Load the library the wrappers call (libmoe_fp8.so unless ``use_library``
    selected another), built by ``fp8_block_scale_gb300.build.build()``."""
    path = _active if path is None else path
    lib = _libs.get(path)
    if lib is not None:
        return lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _libs[path] = lib
    return lib


class use_library:
    """Context manager: the wrappers call the library at `path` (for example
    LIB_DEBUG_PATH, the bounds-checking build) inside the block."""

    def __init__(self, path):
        self.path = path
        self.prev = None

    def __enter__(self):
        global _active
        load(self.path)
        self.prev, _active = _active, self.path
        return _libs[self.path]

    def __exit__(self, *exc):
        global _active
        _active = self.prev
        return False


def moe_debug_bounds_enabled():
    return bool(load().moe_debug_bounds_enabled())


def moe_debug_bounds_selftest(data, probe, out, stream=None):
    """Read data[probe] into out[0] through the bounds checks (int32 device tensors)."""
    _check("moe_debug_bounds_selftest", load().moe_debug_bounds_selftest(
        _ptr(data), data.numel(), int(probe), _ptr(out), _stream(stream)))


def moe_debug_bounds_read(reset=False):
    """(failures, first_file, first_line) of the active library's bounds
    checks since the last reset; waits for the device first."""
    n = ctypes.c_uint64()
    f = ctypes.c_char_p()
    line = ctypes.c_int32()
    _check("moe_debug_bounds_read", load().moe_debug_bounds_read(ctypes.byref(n), ctypes.byref(f),
                                                                 ctypes.byref(line), 1 if reset else 0))
    return n.value, (f.value.decode() if f.value else None), line.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _current_stream():
    # (the raw handle: building a torch.cuda.Stream costs 3 us a call on the Grace host)
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:   # a torch without these names
        return torch.cuda.current_stream().cuda_stream


def _stream(stream=None):
    return ctypes.c_void_p(_current_stream() if stream is None else stream.cuda_stream)


def _check(fn, status):
    if status != MOE_OK:
        raise MoeError(fn, status)


def moe_status_string(status):
    return load().moe_status_string(status).decode()


def moe_plan_capacity(M, top_k, E, block_m):
    cap = ctypes.c_int64()
    blocks = ctypes.c_int64()
    _check("moe_plan_capacity", load().moe_plan_capacity(M, top_k, E, block_m, ctypes.byref(cap), ctypes.byref(blocks)))
    return cap.value, blocks.value


def moe_plan_workspace_size(M, top_k, E):
    return load().moe_plan_workspace_size(M, top_k, E)


def moe_plan(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded, workspace, stream=None):
    M, top_k = topk_ids.shape
    bits = {torch.int32: 32, torch.int64: 64}[topk_ids.dtype]
    _check("moe_plan", load().moe_plan(
        _ptr(topk_ids), bits, M, top_k, E, block_m, _ptr(sorted_token_ids), sorted_token_ids.numel(),
        _ptr(expert_ids), expert_ids.numel(), _ptr(num_tokens_post_padded), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_prep_weights(w13, w13_interleaved, stream=None):
    E, N, H = w13.shape
    _check("moe_prep_weights", load().moe_prep_weights(_ptr(w13), _ptr(w13_interleaved), E, N, H, _stream(stream)))


def moe_requant_scales_ue8m0(w, scale, ue8m0_exp=None, stream=None):
    E, rows, cols = w.shape
    _check("moe_requant_scales_ue8m0", load().moe_requant_scales_ue8m0(
        _ptr(w), _ptr(scale), _ptr(ue8m0_exp), E, rows, cols, _stream(stream)))


LOGITS_F32, LOGITS_BF16 = 0, 1


def moe_route_topk(logits, top_k, topk_ids, topk_weights, routed_scale=1.0, renormalize=True, stream=None):
    """logits [M, E] float32 or bfloat16 -> topk_ids [M, top_k] (int32/int64), topk_weights [M, top_k] f32."""
    M, E = logits.shape
    dtype = {torch.float32: LOGITS_F32, torch.bfloat16: LOGITS_BF16}[logits.dtype]
    bits = {torch.int32: 32, torch.int64: 64}[topk_ids.dtype]
    _check("moe_route_topk", load().moe_route_topk(
        _ptr(logits), dtype, M, E, top_k, float(routed_scale), 1 if renormalize else 0, _ptr(topk_ids), bits,
        _ptr(topk_weights), _stream(stream)))


def moe_route_plan(logits, top_k, topk_ids, topk_weights, block_m, sorted_token_ids, expert_ids,
                   num_tokens_post_padded, routed_scale=1.0, renormalize=True, stream=None):
    """Router and plan in one launch (M * top_k <= 1024, E <= 1024): the
    outputs of moe_route_topk, then of moe_plan on those ids."""
    M, E = logits.shape
    dtype = {torch.float32: LOGITS_F32, torch.bfloat16: LOGITS_BF16}[logits.dtype]
    bits = {torch.int32: 32, torch.int64: 64}[topk_ids.dtype]
    _check("moe_route_plan", load().moe_route_plan(
        _ptr(logits), dtype, M, E, top_k, float(routed_scale), 1 if renormalize else 0, _ptr(topk_ids), bits,
        _ptr(topk_weights), block_m, _ptr(sorted_token_ids), sorted_token_ids.numel(), _ptr(expert_ids),
        expert_ids.numel(), _ptr(num_tokens_post_padded), _stream(stream)))


def moe_quantize_act_1x128(x_bf16, q, scale, stream=None):
    M, H = x_bf16.shape
    _check("moe_quantize_act_1x128", load().moe_quantize_act_1x128(
        _ptr(x_bf16), M, H, _ptr(q), _ptr(scale), _stream(stream)))


def moe_quantize_act_1x128_ue8m0(x_bf16, q, scale, stream=None):
    M, H = x_bf16.shape
    _check("moe_quantize_act_1x128_ue8m0", load().moe_quantize_act_1x128_ue8m0(
        _ptr(x_bf16), M, H, _ptr(q), _ptr(scale), _stream(stream)))


def moe_quantize_weight_128x128(w_bf16, q, scale, stream=None):
    # (BF16, or its bit patterns: another type's bits would be read as BF16)
    if w_bf16.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise ValueError(f"w_bf16: dtype {w_bf16.dtype}, expected {torch.bfloat16}")
    E, rows, cols = w_bf16.shape
    _check("moe_quantize_weight_128x128", load().moe_quantize_weight_128x128(
        _ptr(w_bf16), E, rows, cols, _ptr(q), _ptr(scale), _stream(stream)))


def moe_forward_workspace_size(M, H, I, E, top_k, block_m, sorted_cap):
    return load().moe_forward_workspace_size(M, H, I, E, top_k, block_m, sorted_cap)


def moe_workspace_init(workspace, stream=None):
    _check("moe_workspace_init", load().moe_workspace_init(
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def make_fwd_args(a, a_scale, w13, w13_scale, w2, w2_scale, topk_weights, sorted_token_ids, expert_ids,
                  num_tokens_post_padded, out, workspace, top_k, block_m, routed_scale=1.0,
                  device_status=None, debug_q_inter=None, debug_s_inter=None):
    """Fill a ``moe_fwd_args`` from tensors (shapes give the sizes)."""
    M, H = a.shape
    E, N, _ = w13.shape
    args = MoeFwdArgs()
    args.a, args.a_scale = a.data_ptr(), a_scale.data_ptr()
    args.w13, args.w13_scale = w13.data_ptr(), w13_scale.data_ptr()
    args.w2, args.w2_scale = w2.data_ptr(), w2_scale.data_ptr()
    args.topk_weights = topk_weights.data_ptr()
    args.sorted_token_ids = sorted_token_ids.data_ptr()
    args.expert_ids = expert_ids.data_ptr()
    args.num_tokens_post_padded = num_tokens_post_padded.data_ptr()
    args.out = out.data_ptr()
    args.workspace = workspace.data_ptr()
    args.device_status = device_status.data_ptr() if device_status is not None else None
    args.debug_q_inter = debug_q_inter.data_ptr() if debug_q_inter is not None else None
    args.debug_s_inter = debug_s_inter.data_ptr() if debug_s_inter is not None else None
    args.M = M
    args.sorted_cap = sorted_token_ids.numel()
    args.blocks_cap = expert_ids.numel()
    args.workspace_bytes = workspace.numel() * workspace.element_size()
    args.H, args.I, args.E = H, N // 2, E
    args.top_k, args.block_m = top_k, block_m
    args.routed_scale = routed_scale
    return args


PROFILE_EVENTS = 5  # before staging, after staging, after gate/up, after down, after combine


def set_profile_events(args, events):
    """Attach 5 recorded torch.cuda.Event objects (or None) to a moe_fwd_args."""
    if events is None:
        args.profile_events = None
        args._events_keepalive = None
        return
    if len(events) != PROFILE_EVENTS:
        raise ValueError(f"need {PROFILE_EVENTS} events")
    arr = (ctypes.c_void_p * PROFILE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    args._events_keepalive = arr
    args.profile_events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))


def moe_fp8_block_scale_forward(args, stream=None):
    _check("moe_fp8_block_scale_forward", load().moe_fp8_block_scale_forward(ctypes.byref(args), _stream(stream)))


def moe_selftest_wait_timeout(limit_us, device_status, elapsed_ns, stream=None):
    """Run the bounded-wait self-test; returns the raw status (MOE_ERR_TIMEOUT,
    8, is the expected outcome).  device_status: int32 [1], elapsed_ns:
    int64 [2] device tensors."""
    return load().moe_selftest_wait_timeout(int(limit_us), _ptr(device_status), _ptr(elapsed_ns), _stream(stream))


def moe_noalloc_scratch_bytes():
    return load().moe_noalloc_scratch_bytes()


def moe_fp8_block_scale_forward_noalloc(args, stream=None):
    """Forward without a caller workspace (static device scratch; see the header)."""
    _check("moe_fp8_block_scale_forward_noalloc",
           load().moe_fp8_block_scale_forward_noalloc(ctypes.byref(args), _stream(stream)))


# ---------------------------------------------------------------- E2M1-K32 weights x FP8 activations

def moe_quantize_act_per_row(x_bf16, q, scale, stream=None):
    M, K = x_bf16.shape
    _check("moe_quantize_act_per_row", load().moe_quantize_act_per_row(
        _ptr(x_bf16), M, K, _ptr(q), _ptr(scale), _stream(stream)))


def moe_quantize_weight_k32(w_bf16, q_packed, scale, stream=None):
    """w_bf16 [..., K] (leading dimensions folded into rows) -> q_packed [..., K/2], scale [..., K/32]."""
    K = w_bf16.shape[-1]
    _check("moe_quantize_weight_k32", load().moe_quantize_weight_k32(
        _ptr(w_bf16), w_bf16.numel() // K, K, _ptr(q_packed), _ptr(scale), _stream(stream)))


def moe_w4a8_workspace_size(M, H, I, top_k):
    return load().moe_w4a8_workspace_size(M, H, I, top_k)


def make_w4a8_args(a, a_scale, w13, w13_scale, w2, w2_scale, topk_weights, sorted_token_ids, expert_ids,
                   num_tokens_post_padded, out, workspace, top_k, block_m, routed_scale=1.0,
                   device_status=None, debug_q_inter=None, debug_s_inter=None):
    """Fill a ``moe_w4a8_args`` from tensors; w13 is [E, 2I, H/2] packed codes."""
    M, H = a.shape
    E, N, _ = w13.shape
    args = MoeW4A8Args()
    args.a, args.a_scale = a.data_ptr(), a_scale.data_ptr()
    args.w13, args.w13_scale = w13.data_ptr(), w13_scale.data_ptr()
    args.w2, args.w2_scale = w2.data_ptr(), w2_scale.data_ptr()
    args.topk_weights = topk_weights.data_ptr()
    args.sorted_token_ids = sorted_token_ids.data_ptr()
    args.expert_ids = expert_ids.data_ptr()
    args.num_tokens_post_padded = num_tokens_post_padded.data_ptr()
    args.out = out.data_ptr()
    args.workspace = workspace.data_ptr()
    args.device_status = device_status.data_ptr() if device_status is not None else None
    args.debug_q_inter = debug_q_inter.data_ptr() if debug_q_inter is not None else None
    args.debug_s_inter = debug_s_inter.data_ptr() if debug_s_inter is not None else None
    args.M = M
    args.sorted_cap = sorted_token_ids.numel()
    args.blocks_cap = expert_ids.numel()
    args.workspace_bytes = workspace.numel() * workspace.element_size()
    args.H, args.I, args.E = H, N // 2, E
    args.top_k, args.block_m = top_k, block_m
    args.routed_scale = routed_scale
    return args


def moe_w4a8_forward(args, stream=None):
    _check("moe_w4a8_forward", load().moe_w4a8_forward(ctypes.byref(args), _stream(stream)))


# ---------------------------------------------------------------- training side (include/moe_train.h)
#
# Row buffers may be strided by rows (a slice of wider rows); their elements
# are contiguous within a row.  An argument record keeps the tensors it was made
# from.

def _row_buffer(name, t):
    """(rows, width, row stride) of a 2D row buffer; ValueError if it is not one the library can read."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or stride[1] != 1:
        raise ValueError(f"{name}: a 2D tensor with contiguous rows is expected")
    # (torch gives a single row any stride: no second row follows from it)
    return shape[0], shape[1], stride[0] if shape[0] > 1 else shape[1]


def _rows2d(name, t, dtype=None):
    """(pointer, row stride) of a 2D row buffer."""
    ld = _row_buffer(name, t)[2]
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    return t.data_ptr(), ld


def _dense(name, t, dtype=None, numel=None):
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is expected")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} expected")
    return t.data_ptr()


def _opt(name, t, dtype, numel=None):
    return None if t is None else _dense(name, t, dtype, numel)


def _shape(name, t, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def moe_plan_groups(sorted_token_ids, expert_ids, num_tokens_post_padded, block_m, R, group_start, group_rows,
                    route_slot=None, stream=None):
    """First slot and row count of every expert of a plan (int32 [E] each) and,
    optionally, the slot of every route (int32 [R], -1 where the plan has none)."""
    E = group_start.numel()
    _dense("group_start", group_start, torch.int32)
    _dense("group_rows", group_rows, torch.int32, E)
    _opt("route_slot", route_slot, torch.int32, R)
    _dense("sorted_token_ids", sorted_token_ids, torch.int32)
    _dense("expert_ids", expert_ids, torch.int32)
    _dense("num_tokens_post_padded", num_tokens_post_padded, torch.int32, 1)
    _check("moe_plan_groups", load().moe_plan_groups(
        _ptr(sorted_token_ids), sorted_token_ids.numel(), _ptr(expert_ids), expert_ids.numel(),
        _ptr(num_tokens_post_padded), block_m, R, E, _ptr(group_start), _ptr(group_rows), _ptr(route_slot),
        _stream(stream)))


def moe_gather_rows(x, xs, route_ids, top_k, num_rows=None, stream=None):
    """xs[s] = x[route_ids[s] // top_k]; zero rows where the id is none of the len(x) * top_k routes."""
    M, width, ldx = _row_buffer("x", x)
    rows, w2, ldxs = _row_buffer("xs", xs)
    if width != w2 or x.dtype != xs.dtype:
        raise ValueError("x and xs differ in width or type")
    status = load().moe_gather_rows(
        x.data_ptr(), M, width, ldx, xs.data_ptr(), rows, ldxs, _dense("route_ids", route_ids, torch.int32, rows), top_k,
        None if num_rows is None else _dense("num_rows", num_rows, torch.int32, 1), TYPE_CODES[x.dtype],
        _stream(stream))
    if status:
        raise MoeError("moe_gather_rows", status)


def moe_sum_routes(y, out, route_slot, top_k, accumulate=False, stream=None):
    """out[t] = sum of y[route_slot[t * top_k + j]] over j (on top of out[t] with accumulate)."""
    rows, width, ldy = _row_buffer("y", y)
    M, w2, ldo = _row_buffer("out", out)
    if width != w2 or y.dtype != out.dtype:
        raise ValueError("y and out differ in width or type")
    status = load().moe_sum_routes(
        y.data_ptr(), rows, width, ldy, out.data_ptr(), M, ldo,
        _dense("route_slot", route_slot, torch.int32, M * top_k), top_k, 1 if accumulate else 0, TYPE_CODES[y.dtype],
        _stream(stream))
    if status:
        raise MoeError("moe_sum_routes", status)


def make_grouped_args(x, w, y, group_start, group_rows, input_gradient=False, epilogue=GROUPED_PLAIN, pre=None,
                      route_ids=None, route_weights=None, device_status=None):
    """Fill a ``moe_grouped_args`` from tensors (shapes give the sizes): w [E, N, K];
    x [rows, K] and y [rows, N] (N / 2 with the SwiGLU epilogue), or with
    input_gradient x [rows, N] and y [rows, K]."""
    E, N, K = w.shape
    rows = x.shape[0]
    glu = epilogue == GROUPED_SWIGLU
    args = MoeGroupedArgs()
    args.x, args.ldx = _rows2d("x", x, w.dtype)
    args.y, args.ldy = _rows2d("y", y, w.dtype)
    _shape("x", x, (rows, N if input_gradient else K))
    _shape("y", y, (rows, K if input_gradient else N // 2 if glu else N))
    args.w = _dense("w", w)
    if pre is not None:
        args.pre, args.ldpre = _rows2d("pre", pre, w.dtype)
        _shape("pre", pre, (rows, N))
    args.group_start = _dense("group_start", group_start, torch.int32, E)
    args.group_rows = _dense("group_rows", group_rows, torch.int32, E)
    args.route_ids = _opt("route_ids", route_ids, torch.int32, rows)
    args.route_weights = _opt("route_weights", route_weights, torch.float32, None if route_ids is not None else rows)
    args.device_status = _opt("device_status", device_status, torch.int32, 1)
    args.rows, args.R = rows, 0 if route_weights is None else route_weights.numel()
    args.E, args.N, args.K = E, N, K
    args._keepalive = (x, w, y, group_start, group_rows, pre, route_ids, route_weights, device_status)
    args.dtype = TYPE_CODES[w.dtype]
    args.direction = GROUPED_INPUT_GRADIENT if input_gradient else GROUPED_FORWARD
    args.epilogue = epilogue
    return args


def moe_grouped_gemm(args, stream=None):
    _check("moe_grouped_gemm", load().moe_grouped_gemm(ctypes.byref(args), _stream(stream)))


def make_grouped_wgrad_args(dy, x, dw, group_start, group_rows, accumulate=False, device_status=None):
    """Fill a ``moe_grouped_wgrad_args``: dy [rows, N], x [rows, K], dw [E, N, K] in their type or FP32."""
    E, N, K = dw.shape
    rows = x.shape[0]
    args = MoeGroupedWgradArgs()
    args.dy, args.lddy = _rows2d("dy", dy, x.dtype)
    args.x, args.ldx = _rows2d("x", x)
    _shape("dy", dy, (rows, N))
    _shape("x", x, (rows, K))
    args.dw = _dense("dw", dw)
    args.group_start = _dense("group_start", group_start, torch.int32, E)
    args.group_rows = _dense("group_rows", group_rows, torch.int32, E)
    args.device_status = _opt("device_status", device_status, torch.int32, 1)
    args.rows, args.E, args.N, args.K = rows, E, N, K
    args._keepalive = (dy, x, dw, group_start, group_rows, device_status)
    args.dtype, args.dw_dtype = TYPE_CODES[x.dtype], TYPE_CODES[dw.dtype]
    args.accumulate = 1 if accumulate else 0
    return args


def moe_grouped_wgrad(args, stream=None):
    _check("moe_grouped_wgrad", load().moe_grouped_wgrad(ctypes.byref(args), _stream(stream)))


def make_swiglu_backward_args(dh, pre, dpre, h=None, route_ids=None, num_rows=None, route_weights=None,
                              dweights=None):
    """Fill a ``moe_swiglu_backward_args``: dh and h [rows, I], pre and dpre [rows, 2I]."""
    rows, I = dh.shape
    args = MoeSwigluBackwardArgs()
    args.dh, args.lddh = _rows2d("dh", dh)
    args.pre, args.ldpre = _rows2d("pre", pre, dh.dtype)
    args.dpre, args.lddpre = _rows2d("dpre", dpre, dh.dtype)
    _shape("pre", pre, (rows, 2 * I))
    _shape("dpre", dpre, (rows, 2 * I))
    if h is not None:
        args.h, args.ldh = _rows2d("h", h, dh.dtype)
        _shape("h", h, (rows, I))
    args.route_ids = _opt("route_ids", route_ids, torch.int32, rows)
    args.num_rows = _opt("num_rows", num_rows, torch.int32, 1)
    by_route = [t.numel() for t in (route_weights, dweights) if t is not None]
    need = None if route_ids is not None else rows
    args.route_weights = _opt("route_weights", route_weights, torch.float32, need)
    args.dweights = _opt("dweights", dweights, torch.float32, need)
    # without either, every nonnegative id names a route
    args.R = min(by_route) if by_route else 2 ** 31 - 1
    args._keepalive = (dh, pre, dpre, h, route_ids, num_rows, route_weights, dweights)
    args.rows, args.I, args.dtype = rows, I, TYPE_CODES[dh.dtype]
    return args


def moe_swiglu_backward(args, stream=None):
    _check("moe_swiglu_backward", load().moe_swiglu_backward(ctypes.byref(args), _stream(stream)))


class AdamWTable:
    """The device table of an AdamW step over `tensors`: dicts with ``param``
    (float32), ``grad`` and the states ``exp_avg`` and ``exp_avg_sq``; optionally
    ``model`` (bfloat16 or float16, the rounded copy of param) and
    ``weight_decay`` (the argument's value otherwise).  States are float32, or
    8-bit codes (float8_e4m3fn or uint8) with ``exp_avg_scale`` and
    ``exp_avg_sq_scale``, one float32 per 128 elements.  The table keeps the
    tensors alive."""

    def __init__(self, tensors, weight_decay=0.0, stream=None):
        if not tensors:
            raise ValueError("no tensors")
        self.state_bits = 32 if tensors[0]["exp_avg"].dtype == torch.float32 else 8
        codes = (torch.float32,) if self.state_bits == 32 else (torch.float8_e4m3fn, torch.uint8)
        self.count = len(tensors)
        self.keep = [dict(t) for t in tensors]
        host = (MoeAdamWTensor * self.count)()
        for e, t in zip(host, self.keep):
            n = t["param"].numel()
            e.param = _dense("param", t["param"], torch.float32)
            for name in ("grad", "exp_avg", "exp_avg_sq"):
                setattr(e, name, _dense(name, t[name]))
                if t[name].numel() != n:
                    raise ValueError(f"{name}: {t[name].numel()} elements, expected {n}")
                if name != "grad" and t[name].dtype not in codes:
                    raise ValueError(f"{name}: dtype {t[name].dtype}, expected {codes[0]}")
            model = t.get("model")
            if model is not None:
                e.model = _dense("model", model, None, n)
                e.model_dtype = TYPE_CODES[model.dtype]
            if self.state_bits == 8:
                e.exp_avg_scale = _dense("exp_avg_scale", t["exp_avg_scale"], torch.float32, -(-n // 128))
                e.exp_avg_sq_scale = _dense("exp_avg_sq_scale", t["exp_avg_sq_scale"], torch.float32, -(-n // 128))
            e.n = n
            e.grad_dtype = TYPE_CODES[t["grad"].dtype]
            e.weight_decay = float(t.get("weight_decay", weight_decay))
        lib = load()
        self.table = torch.empty(lib.moe_adamw_table_bytes(self.count), dtype=torch.uint8,
                                 device=tensors[0]["param"].device)
        chunks, types = ctypes.c_int64(), ctypes.c_int32()
        _check("moe_adamw_table_init", lib.moe_adamw_table_init(
            host, self.count, self.state_bits, _ptr(self.table), self.table.numel(), ctypes.byref(chunks),
            ctypes.byref(types), _stream(stream)))
        self.chunks, self.grad_types = chunks.value, types.value


def make_adamw_args(table, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, seed=0, grad_scale=None, skip=None):
    """Fill a ``moe_adamw_args`` for an AdamWTable; lr, step and seed are the
    fields a loop rewrites between steps."""
    args = MoeAdamWArgs()
    args._table_keepalive = (table, grad_scale, skip)
    args.table, args.chunks, args.count = table.table.data_ptr(), table.chunks, table.count
    args.state_bits, args.grad_types = table.state_bits, table.grad_types
    args.grad_scale = _opt("grad_scale", grad_scale, torch.float32, 1)
    args.skip = _opt("skip", skip, torch.int32, 1)
    args.lr, args.step, args.beta1, args.beta2, args.eps, args.seed = lr, step, beta1, beta2, eps, seed & 0xFFFFFFFF
    return args


def moe_adamw_step(args, stream=None):
    _check("moe_adamw_step", load().moe_adamw_step(ctypes.byref(args), _stream(stream)))


# ---------------------------------------------------------------- around the experts (include/moe_block.h)
#
# Row buffers and argument records as on the training side.

ID_BITS = {torch.int32: 32, torch.int64: 64}


def _code(name, t, codes, names):
    if t.dtype not in codes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {names}")
    return codes[t.dtype]


def _logits(name, t):
    """(pointer, M, E, elements from a row to the next, type) of router logits."""
    M, E, ld = _row_buffer(name, t)
    return t.data_ptr(), M, E, ld, _code(name, t, TYPE_CODES, "bfloat16, float16 or float32")


def _routes(ids, other_name, other, M):
    """top_k and id width of a token's routes: ids [M, top_k] and a float32 tensor of that shape."""
    if len(ids.shape) != 2 or ids.shape[0] != M:
        raise ValueError(f"topk_ids: shape {tuple(ids.shape)}, expected ({M}, top_k)")
    _dense("topk_ids", ids)
    _dense(other_name, other, torch.float32)
    _shape(other_name, other, ids.shape)
    return ids.shape[1], _code("topk_ids", ids, ID_BITS, "int32 or int64")


def make_route_scores_args(logits, topk_ids, topk_weights, bias=None, score=SCORE_SIGMOID, groups=1, topk_groups=1,
                           group_score=GROUP_MAX, renormalize=True, routed_scale=1.0, num_tokens=None):
    """Fill a ``moe_route_scores_args``: logits [M, E] (bfloat16, float16 or float32), topk_ids
    [M, top_k] int32 or int64, topk_weights [M, top_k] and bias [E] float32, num_tokens [1] int32."""
    args = MoeRouteScoresArgs()
    args.logits, args.M, args.E, args.ldlogits, args.dtype = _logits("logits", logits)
    args.top_k, args.id_bits = _routes(topk_ids, "topk_weights", topk_weights, args.M)
    args.topk_ids, args.topk_weights = topk_ids.data_ptr(), topk_weights.data_ptr()
    if bias is not None:
        _shape("bias", bias, (args.E,))
    args.bias = _opt("bias", bias, torch.float32)
    args.num_tokens = _opt("num_tokens", num_tokens, torch.int32, 1)
    args.groups, args.topk_groups, args.group_score, args.score = groups, topk_groups, group_score, score
    args.renormalize, args.routed_scale = 1 if renormalize else 0, routed_scale
    args._keepalive = (logits, topk_ids, topk_weights, bias, num_tokens)
    return args


def moe_route_scores(args, stream=None):
    _check("moe_route_scores", load().moe_route_scores(ctypes.byref(args), _stream(stream)))


def make_route_scores_backward_args(logits, topk_ids, dweights, dlogits, score=SCORE_SIGMOID, renormalize=True,
                                    routed_scale=1.0, num_tokens=None):
    """Fill a ``moe_route_scores_backward_args``: dlogits of logits' shape and type (it may be logits)."""
    args = MoeRouteScoresBackwardArgs()
    args.logits, args.M, args.E, args.ldlogits, args.dtype = _logits("logits", logits)
    args.dlogits, args.lddlogits = _rows2d("dlogits", dlogits, logits.dtype)
    _shape("dlogits", dlogits, logits.shape)
    args.top_k, args.id_bits = _routes(topk_ids, "dweights", dweights, args.M)
    args.topk_ids, args.dweights = topk_ids.data_ptr(), dweights.data_ptr()
    args.num_tokens = _opt("num_tokens", num_tokens, torch.int32, 1)
    args.score, args.renormalize, args.routed_scale = score, 1 if renormalize else 0, routed_scale
    args._keepalive = (logits, topk_ids, dweights, dlogits, num_tokens)
    return args


def moe_route_scores_backward(args, stream=None):
    _check("moe_route_scores_backward", load().moe_route_scores_backward(ctypes.byref(args), _stream(stream)))


def moe_route_balance(load_of_experts, bias, rate, out=None, stream=None):
    """bias [E] float32 (or out, without touching bias) one step of `rate` towards an even load
    (load_of_experts [E] int32, for example a plan's group_rows)."""
    out = bias if out is None else out
    E = bias.numel()
    _dense("bias", bias, torch.float32)
    _dense("out", out, torch.float32)
    _dense("load_of_experts", load_of_experts, torch.int32)
    for name, t in (("out", out), ("load_of_experts", load_of_experts)):
        if t.numel() != E:
            raise ValueError(f"{name}: {t.numel()} elements, expected {E}")
    _check("moe_route_balance", load().moe_route_balance(_ptr(load_of_experts), _ptr(bias), _ptr(out), E, rate,
                                                         _stream(stream)))


def _norm_common(args, y, gate, w_post, w_pre, post_norm, residual_scale, weight_offset, eps, num_rows):
    """The fields both directions share; returns (branch type, its shape)."""
    M, H, args.ldy = _row_buffer("y", y)
    args.y, args.M, args.H = y.data_ptr(), M, H
    args.dtype = _code("y", y, TYPE_CODES, "bfloat16, float16 or float32")
    weights = [(n, w) for n, w in (("w_post", w_post), ("w_pre", w_pre)) if w is not None]
    if w_post is not None and not post_norm:
        raise ValueError("w_post: given without post_norm")
    mode = GATE_NONE
    if gate is not None:
        shape = tuple(gate.shape)
        if shape == (M, H):
            mode = GATE_FULL
            args.gate, args.ldgate = _rows2d("gate", gate, y.dtype)
        elif shape == (M, 1):
            mode = GATE_TOKEN
            args.gate = _dense("gate", gate, torch.float32)
        elif shape == (H,):
            mode = GATE_CHANNEL
            args.gate = _dense("gate", gate)
            weights.append(("gate", gate))
        else:
            raise ValueError(f"gate: shape {shape}, expected ({H},), ({M}, 1) or ({M}, {H})")
    kind = weights[0][1].dtype if weights else y.dtype
    for name, w in weights:
        _shape(name, w, (H,))
        if w.dtype != kind or kind not in (y.dtype, torch.float32):
            raise ValueError(f"{name}: dtype {w.dtype}, expected one type for weights and channel gate, {y.dtype} or float32")
    args.w_post, args.w_pre = _opt("w_post", w_post, kind), _opt("w_pre", w_pre, kind)
    args.weight_dtype, args.gate_mode, args.post_norm = TYPE_CODES[kind], mode, 1 if post_norm else 0
    args.residual_scale, args.weight_offset, args.eps = residual_scale, weight_offset, eps
    args.num_rows = _opt("num_rows", num_rows, torch.int32, 1)
    return M, H


def _stream_rows(args, y, tensors):
    """The residual stream's buffers: one type, y's or float32."""
    kind = None
    for name, t, field, ld in tensors:
        if t is None:
            continue
        kind = t.dtype if kind is None else kind
        if t.dtype != kind or kind not in (y.dtype, torch.float32):
            raise ValueError(f"{name}: dtype {t.dtype}, expected one type for the stream, {y.dtype} or float32")
        _shape(name, t, y.shape)
        p, stride = _rows2d(name, t)
        setattr(args, field, p)
        setattr(args, ld, stride)
    args.stream_dtype = TYPE_CODES[y.dtype if kind is None else kind]


def _branch_rows(args, y, tensors):
    for name, t, field, ld in tensors:
        if t is not None:
            _shape(name, t, y.shape)
            p, stride = _rows2d(name, t, y.dtype)
            setattr(args, field, p)
            setattr(args, ld, stride)


def make_norm_residual_args(y, h=None, z=None, r=None, gate=None, w_post=None, w_pre=None, post_norm=None,
                            residual_scale=1.0, eps=1e-6, weight_offset=0.0, q=None, q_scale=None,
                            scale_mode=SCALES_FP32, num_rows=None):
    """Fill a ``moe_norm_args`` from tensors: the branch y [M, H], the stream r and h (y's type or
    float32), z like y, q [M, H] (float8_e4m3fn or uint8) with q_scale [M, H / 128].

    gate: [H] one for each channel (the weights' type), [M, 1] one for each token (float32), [M, H]
    (y's type).  post_norm: the branch is normed (w_post None: weight 1); by default it is where
    w_post is given."""
    args = MoeNormArgs()
    M, H = _norm_common(args, y, gate, w_post, w_pre, w_post is not None if post_norm is None else post_norm, residual_scale,
                        weight_offset, eps, num_rows)
    _stream_rows(args, y, (("r", r, "r", "ldr"), ("h", h, "h", "ldh")))
    _branch_rows(args, y, (("z", z, "z", "ldz"),))
    if (q is None) != (q_scale is None):
        raise ValueError("q and q_scale go together")
    if q is not None:
        if q.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError(f"q: dtype {q.dtype}, expected {torch.float8_e4m3fn}")
        _shape("q", q, (M, H))
        _shape("q_scale", q_scale, (M, H // 128))
        args.q, args.q_scale = _dense("q", q), _dense("q_scale", q_scale, torch.float32)
    args.scale_mode = scale_mode
    args._keepalive = (y, h, z, r, gate, w_post, w_pre, q, q_scale, num_rows)
    return args


def moe_norm_residual(args, stream=None):
    _check("moe_norm_residual", load().moe_norm_residual(ctypes.byref(args), _stream(stream)))


def moe_norm_residual_workspace_size(M, H):
    return load().moe_norm_residual_workspace_size(M, H)


def make_norm_residual_backward_args(y, dh=None, dz=None, h=None, gate=None, w_post=None, w_pre=None, post_norm=None,
                                     residual_scale=1.0, eps=1e-6, weight_offset=0.0, dy=None, dr=None, dgate=None,
                                     dw_post=None, dw_pre=None, workspace=None, accumulate=False, num_rows=None):
    """Fill a ``moe_norm_backward_args``: the forward's y, h, gate and weights, the gradients dh (at h,
    from the stream) and dz that arrive, and those asked for.  dw_post, dw_pre and a channel gate's
    dgate are float32 [H], a token gate's float32 of its shape, a full one's like y."""
    args = MoeNormBackwardArgs()
    M, H = _norm_common(args, y, gate, w_post, w_pre, w_post is not None if post_norm is None else post_norm, residual_scale,
                        weight_offset, eps, num_rows)
    _stream_rows(args, y, (("h", h, "h", "ldh"), ("dh", dh, "dh", "lddh"), ("dr", dr, "dr", "lddr")))
    _branch_rows(args, y, (("dz", dz, "dz", "lddz"), ("dy", dy, "dy", "lddy")))
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate: given without a gate")
        _shape("dgate", dgate, gate.shape)
        if args.gate_mode == GATE_FULL:
            args.dgate, args.lddgate = _rows2d("dgate", dgate, y.dtype)
        else:
            args.dgate = _dense("dgate", dgate, torch.float32)
    for name, t in (("dw_post", dw_post), ("dw_pre", dw_pre)):
        if t is not None:
            _shape(name, t, (H,))
    args.dw_post, args.dw_pre = _opt("dw_post", dw_post, torch.float32), _opt("dw_pre", dw_pre, torch.float32)
    if workspace is not None:
        args.workspace = _dense("workspace", workspace)
        args.workspace_bytes = workspace.numel() * workspace.element_size()
    args.accumulate = 1 if accumulate else 0
    args._keepalive = (y, dh, dz, h, gate, w_post, w_pre, dy, dr, dgate, dw_post, dw_pre, workspace, num_rows)
    return args


def moe_norm_residual_backward(args, stream=None):
    _check("moe_norm_residual_backward", load().moe_norm_residual_backward(ctypes.byref(args), _stream(stream)))
