"""ctypes binding of libfp4lin (argument marshalling only).

Every function here has the name and argument order of the C entry point
declared in include/fp4lin.h.  Tensor arguments may be torch tensors (their
data pointers are passed), plain integers (raw device pointers) or None
(NULL).  `stream` defaults to torch's current CUDA stream.  A non-OK status
raises Fp4Error.  There is no fallback: if the library is missing or the
GPU is not sm_103, calls fail.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4lin.so")

FP4_OK = 0
FP4_ERR_INVALID_ARG = 1
FP4_ERR_SHAPE = 2
FP4_ERR_ALIGNMENT = 3
FP4_ERR_UNSUPPORTED = 4
FP4_ERR_CUDA = 5
FP4_ERR_TIMEOUT = 6
FP4_SCALE_OCP = 0
FP4_SCALE_UOS = 2
FP4_SF_SWIZZLED = 0
FP4_SF_ROWMAJOR = 1

# every symbol the header declares
SYMBOLS = (
    "fp4_sf_bytes", "fp4_sf_bytes_grouped", "fp4_status_string", "fp4_get_device_status",
    "fp4_requant_nvfp4_to_mxfp4", "fp4_requant_nvfp4_to_mxfp4_ex", "fp4_requant_nvfp4_to_mxfp4_grouped",
    "fp4_quant_act_mxfp4",
    "fp4_quant_act_mxfp4_grouped", "fp4_quant_nvfp4", "fp4_gemm_mxfp4", "fp4_gemm_workspace_size",
    "fp4_gemm_mxfp4_ws", "fp4_gemm_mxfp4_noalloc", "fp4_gemm_mxfp4_grouped",
    "fp4_quant_nvfp4_ex", "fp4_sf_bytes_nvfp4", "fp4_sf_swizzle", "fp4_gemm_nvfp4",
    "fp4_quant_act_mxfp8", "fp4_gemm_w4a8", "fp4_gemm_w4a8_workspace_size", "fp4_gemm_mxfp4_ex",
    "fp4_smooth_prepare", "fp4_quant_act_mxfp4_smooth", "fp4_quant_act_mxfp8_smooth",
    "fp4_linear_workspace_size", "fp4_linear", "fp4_linear_grouped_workspace_size", "fp4_linear_grouped",
    "fp4_debug_set_wait_fault", "fp4_quant_dualscale", "fp4_gemm_mxfp4_dualscale",
    "fp4_fp8_act_scale_bytes", "fp4_quant_act_fp8_b128", "fp4_quant_weight_fp8_b128", "fp4_gemm_fp8_b128",
    "fp4_linear_fp8_b128_workspace_size", "fp4_linear_fp8_b128", "fp4_rope_table", "fp4_rope",
    "fp4_kv_code_bytes", "fp4_kv_scale_bytes", "fp4_kv_append", "fp4_kv_read",
    "fp4_kv_attention_workspace_size", "fp4_kv_attention",
)


class Fp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)}")
        self.status = status


class fp4_quant_opts(ctypes.Structure):
    _fields_ = [("scale_alg", ctypes.c_int32), ("sf_layout", ctypes.c_int32), ("flags", ctypes.c_uint32)]


FP4_QUANT_BF16_INTERMEDIATE = 1


class fp4_linear_opts(ctypes.Structure):
    _fields_ = [("act_format", ctypes.c_int32), ("scale_alg", ctypes.c_int32), ("mul_scale_bf16", ctypes.c_void_p),
                ("gemm_flags", ctypes.c_uint32)]


FP4_ACT_MXFP4 = 0
FP4_ACT_MXFP8 = 1
FP4_LINEAR_FUSED_QUANT = 2

FP4_ROPE_HALF = 0
FP4_ROPE_INTERLEAVED = 1
FP4_ROPE_INVERSE = 1
FP4_ROPE_UNSCALED = 0
FP4_ROPE_LINEAR = 1
FP4_ROPE_BY_PARTS = 2


class fp4_rope_params(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_positions", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class fp4_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_positions", ctypes.c_int64),
                ("turns_fast", ctypes.c_double), ("turns_slow", ctypes.c_double), ("magnitude", ctypes.c_double)]


class fp4_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class fp4_kv_attention_args(ctypes.Structure):
    _fields_ = [("q_bf16", ctypes.c_void_p), ("out_bf16", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
                ("context_lens", ctypes.c_void_p), ("q_offsets", ctypes.c_void_p), ("tree_mask", ctypes.c_void_p),
                ("mask_words", ctypes.c_int32), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int32), ("max_draft", ctypes.c_int32), ("max_seq_len", ctypes.c_int64),
                ("softmax_scale", ctypes.c_float)]


# the same layout in one step: the structure's constructor costs as much as the checks of a call
_attention_args = struct.Struct("@PPPqqqqPqPPPiiqiiqf4x").pack


_lib = None
_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32


def load(path: str = LIB_PATH):
    """Loads the shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise FileNotFoundError(f"{path} is missing: build it with nvfp4_mxfp4_w4a4_gb300.build.build()")
        L = ctypes.CDLL(path)
        sig = {
            "fp4_sf_bytes": (ctypes.c_size_t, [_i64, _i64, _i32]),
            "fp4_sf_bytes_grouped": (ctypes.c_size_t, [_i64, _i32, _i64]),
            "fp4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "fp4_get_device_status": (ctypes.c_int, []),
            "fp4_debug_set_wait_fault": (ctypes.c_int, [ctypes.c_uint64, _i32]),
            "fp4_quant_dualscale": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i64, _i32, _p]),
            "fp4_gemm_mxfp4_dualscale": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p,
                                                        ctypes.c_size_t, _p]),
            "fp4_requant_nvfp4_to_mxfp4": (ctypes.c_int, [_p, _p, ctypes.c_float, _p, _p, _i64, _i64, _p]),
            "fp4_requant_nvfp4_to_mxfp4_ex": (ctypes.c_int, [_p, _p, ctypes.c_float, _p, _p, _i64, _i64,
                                                             ctypes.POINTER(fp4_quant_opts), _p]),
            "fp4_requant_nvfp4_to_mxfp4_grouped": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64,
                                                                  ctypes.POINTER(fp4_quant_opts), _p]),
            "fp4_quant_act_mxfp4": (ctypes.c_int, [_p, _p, _p, _i64, _i64, ctypes.POINTER(fp4_quant_opts), _p]),
            "fp4_quant_act_mxfp4_grouped": (ctypes.c_int, [_p, _p, _i32, _i64, _i64, _p, _p,
                                                           ctypes.POINTER(fp4_quant_opts), _p]),
            "fp4_quant_nvfp4": (ctypes.c_int, [_p, ctypes.c_float, _p, _p, _i64, _i64, _p]),
            "fp4_gemm_mxfp4": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
            "fp4_gemm_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64]),
            "fp4_gemm_mxfp4_ws": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_size_t, _p]),
            "fp4_gemm_mxfp4_noalloc": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
            "fp4_gemm_mxfp4_grouped": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p]),
            "fp4_quant_nvfp4_ex": (ctypes.c_int, [_p, ctypes.c_float, _p, _p, _i64, _i64, _i32, _p]),
            "fp4_sf_bytes_nvfp4": (ctypes.c_size_t, [_i64, _i64, _i32]),
            "fp4_sf_swizzle": (ctypes.c_int, [_p, _p, _i64, _i64, _p]),
            "fp4_gemm_nvfp4": (ctypes.c_int, [_p, _p, _p, _p, ctypes.c_float, _p, _p, _i64, _i64, _i64, _p,
                                              ctypes.c_size_t, _p]),
            "fp4_quant_act_mxfp8": (ctypes.c_int, [_p, _p, _p, _i64, _i64, _i32, _p]),
            "fp4_gemm_w4a8": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_size_t, _p]),
            "fp4_gemm_w4a8_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64]),
            "fp4_gemm_mxfp4_ex": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_size_t,
                                                 ctypes.c_uint32, _p]),
            "fp4_smooth_prepare": (ctypes.c_int, [_p, _p, _i64, _p, _p]),
            "fp4_quant_act_mxfp4_smooth": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i64,
                                                          ctypes.POINTER(fp4_quant_opts), _p]),
            "fp4_quant_act_mxfp8_smooth": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i64, _i32, _p]),
            "fp4_linear_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, ctypes.POINTER(fp4_linear_opts)]),
            "fp4_linear": (ctypes.c_int, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_size_t,
                                          ctypes.POINTER(fp4_linear_opts), _p]),
            "fp4_fp8_act_scale_bytes": (ctypes.c_size_t, [_i64, _i64]),
            "fp4_quant_act_fp8_b128": (ctypes.c_int, [_p, _p, _p, _i64, _i64, _p]),
            "fp4_quant_weight_fp8_b128": (ctypes.c_int, [_p, _p, _p, _i64, _i64, _p]),
            "fp4_gemm_fp8_b128": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p]),
            "fp4_linear_fp8_b128_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64]),
            "fp4_linear_fp8_b128": (ctypes.c_int, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_size_t, _p]),
            "fp4_rope_table": (ctypes.c_int, [_p, _i64, _i32, ctypes.c_double, ctypes.POINTER(fp4_rope_scaling), _p]),
            "fp4_rope": (ctypes.c_int, [_p, _p, _p, ctypes.POINTER(fp4_rope_params), _i64, _i32, _i32, _i64, _i64, _i64,
                                        _i64, _p]),
            "fp4_kv_code_bytes": (ctypes.c_size_t, [ctypes.POINTER(fp4_kv_cache)]),
            "fp4_kv_scale_bytes": (ctypes.c_size_t, [ctypes.POINTER(fp4_kv_cache)]),
            "fp4_kv_append": (ctypes.c_int, [ctypes.POINTER(fp4_kv_cache), _p, _p, _i64, _i64, _i64, _i64, _i64, _p,
                                             ctypes.POINTER(fp4_rope_params), _p, _p]),
            "fp4_kv_read": (ctypes.c_int, [ctypes.POINTER(fp4_kv_cache), _p, _i64, _p, _i32, _i64, _p, _p, _p]),
            "fp4_kv_attention_workspace_size": (ctypes.c_size_t, [_i32, _i64, _i32, _i32, _i32, _i64, _i32]),
            "fp4_kv_attention": (ctypes.c_int, [ctypes.POINTER(fp4_kv_cache), _p, _p,
                                                ctypes.c_size_t, _p]),
            "fp4_linear_grouped_workspace_size": (ctypes.c_size_t, [_i64, _i32, _i64]),
            "fp4_linear_grouped": (ctypes.c_int, [_p, _p, _i32, _i64, _p, _p, _p, _p, _i64, _i64, _p, ctypes.c_size_t,
                                                  ctypes.POINTER(fp4_quant_opts), _p]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(s):
    global _current_stream
    if s is None:
        if _current_stream is None:
            import torch

            # the handle alone, where this torch has it: the Stream object that
            # torch.cuda.current_stream() builds costs as much as a launch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            dev = getattr(torch._C, "_cuda_getDevice", None)
            torch.cuda.init()
            _current_stream = (lambda: raw(dev())) if raw and dev else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _opts(scale_alg, sf_layout, flags=0):
    if scale_alg is None and sf_layout is None and not flags:
        return None
    o = fp4_quant_opts(FP4_SCALE_OCP if scale_alg is None else scale_alg,
                       FP4_SF_SWIZZLED if sf_layout is None else sf_layout, flags)
    return ctypes.byref(o)


def _check(status: int, where: str):
    if status != FP4_OK:
        raise Fp4Error(status, where)


def status_string(status: int) -> str:
    return load().fp4_status_string(status).decode()


def fp4_sf_bytes(rows: int, K: int, sf_layout: int = FP4_SF_SWIZZLED) -> int:
    return load().fp4_sf_bytes(rows, K, sf_layout)


def fp4_sf_bytes_grouped(total_M: int, E: int, K: int) -> int:
    return load().fp4_sf_bytes_grouped(total_M, E, K)


def fp4_get_device_status() -> int:
    return load().fp4_get_device_status()


def fp4_debug_set_wait_fault(wait_limit_ns: int = 0, withhold_split_signal: int = 0):
    """Test hook: limit of the GEMMs' bounded device waits (0 = the default
    1 s) and whether a split-K partial withholds its ready signal."""
    _check(load().fp4_debug_set_wait_fault(wait_limit_ns, withhold_split_signal), "fp4_debug_set_wait_fault")


def fp4_requant_nvfp4_to_mxfp4(w_packed, w_scale_e4m3, w_global, out_packed, out_scale, N, K, stream=None,
                               scale_alg=None, sf_layout=None, bf16_intermediate=False):
    """bf16_intermediate: round each decoded value to bf16 before the block rule."""
    L = load()
    flags = FP4_QUANT_BF16_INTERMEDIATE if bf16_intermediate else 0
    if scale_alg is None and sf_layout is None and not flags:
        st = L.fp4_requant_nvfp4_to_mxfp4(_ptr(w_packed), _ptr(w_scale_e4m3), float(w_global), _ptr(out_packed),
                                          _ptr(out_scale), N, K, _stream(stream))
    else:
        st = L.fp4_requant_nvfp4_to_mxfp4_ex(_ptr(w_packed), _ptr(w_scale_e4m3), float(w_global),
                                             _ptr(out_packed), _ptr(out_scale), N, K,
                                             _opts(scale_alg, sf_layout, flags), _stream(stream))
    _check(st, "fp4_requant_nvfp4_to_mxfp4")


def fp4_requant_nvfp4_to_mxfp4_grouped(w_packed, w_scale_e4m3, w_global, out_packed, out_scale, E, N, K,
                                       stream=None, scale_alg=None, sf_layout=None, bf16_intermediate=False):
    """w_global: device array of E float32 global scales."""
    flags = FP4_QUANT_BF16_INTERMEDIATE if bf16_intermediate else 0
    st = load().fp4_requant_nvfp4_to_mxfp4_grouped(_ptr(w_packed), _ptr(w_scale_e4m3), _ptr(w_global),
                                                   _ptr(out_packed), _ptr(out_scale), E, N, K,
                                                   _opts(scale_alg, sf_layout, flags), _stream(stream))
    _check(st, "fp4_requant_nvfp4_to_mxfp4_grouped")


def fp4_quant_act_mxfp4(x_bf16, out_packed, out_scale, M, K, stream=None, scale_alg=None, sf_layout=None):
    st = load().fp4_quant_act_mxfp4(_ptr(x_bf16), _ptr(out_packed), _ptr(out_scale), M, K,
                                    _opts(scale_alg, sf_layout), _stream(stream))
    _check(st, "fp4_quant_act_mxfp4")


def fp4_quant_act_mxfp4_grouped(x_bf16, row_offsets, E, total_M, K, out_packed, out_scale, stream=None,
                                scale_alg=None):
    st = load().fp4_quant_act_mxfp4_grouped(_ptr(x_bf16), _ptr(row_offsets), E, total_M, K, _ptr(out_packed),
                                            _ptr(out_scale), _opts(scale_alg, None), _stream(stream))
    _check(st, "fp4_quant_act_mxfp4_grouped")


def fp4_quant_nvfp4(x_bf16, g, out_packed, out_scale_e4m3, M, K, stream=None):
    st = load().fp4_quant_nvfp4(_ptr(x_bf16), float(g), _ptr(out_packed), _ptr(out_scale_e4m3), M, K,
                                _stream(stream))
    _check(st, "fp4_quant_nvfp4")


def fp4_quant_nvfp4_ex(x_bf16, g, out_packed, out_scale_e4m3, M, K, sf_layout=FP4_SF_SWIZZLED, stream=None):
    st = load().fp4_quant_nvfp4_ex(_ptr(x_bf16), float(g), _ptr(out_packed), _ptr(out_scale_e4m3), M, K, sf_layout,
                                   _stream(stream))
    _check(st, "fp4_quant_nvfp4_ex")


def fp4_sf_bytes_nvfp4(rows: int, K: int, sf_layout: int = FP4_SF_SWIZZLED) -> int:
    return load().fp4_sf_bytes_nvfp4(rows, K, sf_layout)


def fp4_sf_swizzle(in_rowmajor, out, rows, kblocks, stream=None):
    st = load().fp4_sf_swizzle(_ptr(in_rowmajor), _ptr(out), rows, kblocks, _stream(stream))
    _check(st, "fp4_sf_swizzle")


def fp4_gemm_nvfp4(a, sa, b, sb, alpha, bias_bf16, out_bf16, M, N, K, workspace=None, workspace_bytes=None,
                   stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().fp4_gemm_nvfp4(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), float(alpha), _ptr(bias_bf16), _ptr(out_bf16),
                               M, N, K, _ptr(workspace), workspace_bytes, _stream(stream))
    _check(st, "fp4_gemm_nvfp4")


def fp4_quant_act_mxfp8(x_bf16, out_e4m3, out_scale, M, K, sf_layout=FP4_SF_SWIZZLED, stream=None):
    st = load().fp4_quant_act_mxfp8(_ptr(x_bf16), _ptr(out_e4m3), _ptr(out_scale), M, K, sf_layout,
                                    _stream(stream))
    _check(st, "fp4_quant_act_mxfp8")


def fp4_smooth_prepare(mul_scale_f32, out_bf16, K, bad_count, stream=None):
    """Converts the float32 smooth tensor to bf16; bad_count (device int32)
    receives the number of values that loading must reject."""
    st = load().fp4_smooth_prepare(_ptr(mul_scale_f32), _ptr(out_bf16), K, _ptr(bad_count), _stream(stream))
    _check(st, "fp4_smooth_prepare")


def fp4_quant_act_mxfp4_smooth(x_bf16, mul_scale_bf16, out_packed, out_scale, M, K, stream=None, scale_alg=None,
                               sf_layout=None):
    st = load().fp4_quant_act_mxfp4_smooth(_ptr(x_bf16), _ptr(mul_scale_bf16), _ptr(out_packed), _ptr(out_scale),
                                           M, K, _opts(scale_alg, sf_layout), _stream(stream))
    _check(st, "fp4_quant_act_mxfp4_smooth")


def fp4_quant_act_mxfp8_smooth(x_bf16, mul_scale_bf16, out_e4m3, out_scale, M, K, sf_layout=FP4_SF_SWIZZLED,
                               stream=None):
    st = load().fp4_quant_act_mxfp8_smooth(_ptr(x_bf16), _ptr(mul_scale_bf16), _ptr(out_e4m3), _ptr(out_scale), M,
                                           K, sf_layout, _stream(stream))
    _check(st, "fp4_quant_act_mxfp8_smooth")


def _linear_opts(act_format, scale_alg, mul_scale_bf16, gemm_flags):
    return fp4_linear_opts(act_format, scale_alg, _ptr(mul_scale_bf16), gemm_flags)


def fp4_linear_workspace_size(M, N, K, act_format=FP4_ACT_MXFP4, scale_alg=FP4_SCALE_OCP, mul_scale_bf16=None,
                              gemm_flags=0) -> int:
    o = _linear_opts(act_format, scale_alg, mul_scale_bf16, gemm_flags)
    return load().fp4_linear_workspace_size(M, N, K, ctypes.byref(o))


def fp4_linear(x_bf16, w, sw, bias_bf16, out_bf16, M, N, K, workspace, workspace_bytes=None,
               act_format=FP4_ACT_MXFP4, scale_alg=FP4_SCALE_OCP, mul_scale_bf16=None, gemm_flags=0, stream=None):
    """y = quant(x [* mul_scale]) . W^T (+ bias) in one call; workspace from
    fp4_linear_workspace_size, zeroed once before first use."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    o = _linear_opts(act_format, scale_alg, mul_scale_bf16, gemm_flags)
    st = load().fp4_linear(_ptr(x_bf16), _ptr(w), _ptr(sw), _ptr(bias_bf16), _ptr(out_bf16), M, N, K, _ptr(workspace),
                           workspace_bytes, ctypes.byref(o), _stream(stream))
    _check(st, "fp4_linear")


def fp4_linear_grouped_workspace_size(total_M, E, K) -> int:
    return load().fp4_linear_grouped_workspace_size(total_M, E, K)


def fp4_linear_grouped(x_bf16, row_offsets, E, total_M, w, sw, bias_bf16, out_bf16, N, K, workspace,
                       workspace_bytes=None, scale_alg=None, stream=None):
    """MoE form of fp4_linear: grouped act-quant then grouped GEMM."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = load().fp4_linear_grouped(_ptr(x_bf16), _ptr(row_offsets), E, total_M, _ptr(w), _ptr(sw), _ptr(bias_bf16),
                                   _ptr(out_bf16), N, K, _ptr(workspace), workspace_bytes, _opts(scale_alg, None),
                                   _stream(stream))
    _check(st, "fp4_linear_grouped")


def fp4_gemm_w4a8_workspace_size(M, N, K) -> int:
    return load().fp4_gemm_w4a8_workspace_size(M, N, K)


def fp4_gemm_w4a8(a_e4m3, sa, b, sb, bias_bf16, out_bf16, M, N, K, workspace=None, workspace_bytes=None,
                  stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().fp4_gemm_w4a8(_ptr(a_e4m3), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                              _ptr(workspace), workspace_bytes, _stream(stream))
    _check(st, "fp4_gemm_w4a8")


def fp4_gemm_mxfp4(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, stream=None):
    st = load().fp4_gemm_mxfp4(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                               _stream(stream))
    _check(st, "fp4_gemm_mxfp4")


def fp4_gemm_workspace_size(M, N, K) -> int:
    return load().fp4_gemm_workspace_size(M, N, K)


def fp4_gemm_mxfp4_ws(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, workspace, workspace_bytes=None, stream=None):
    """workspace: device buffer (e.g. a zero-initialised uint8 tensor) or None."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().fp4_gemm_mxfp4_ws(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                                  _ptr(workspace), workspace_bytes, _stream(stream))
    _check(st, "fp4_gemm_mxfp4_ws")


FP4_GEMM_WEIGHTS_STATIC = 1


def fp4_gemm_mxfp4_ex(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, workspace=None, workspace_bytes=None, flags=0,
                      stream=None):
    """flags: FP4_GEMM_WEIGHTS_STATIC when b / sb are not written by the kernel
    enqueued just before this call (the GEMM then streams its first weight
    stages while that kernel finishes)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().fp4_gemm_mxfp4_ex(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                                  _ptr(workspace), workspace_bytes, flags, _stream(stream))
    _check(st, "fp4_gemm_mxfp4_ex")


def fp4_gemm_mxfp4_noalloc(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, stream=None):
    """The GEMM with the library's fixed device scratch (allocates nothing)."""
    st = load().fp4_gemm_mxfp4_noalloc(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N,
                                       K, _stream(stream))
    _check(st, "fp4_gemm_mxfp4_noalloc")


def fp4_gemm_mxfp4_grouped(a, sa, b, sb, bias_bf16, out_bf16, row_offsets, E, total_M, N, K, stream=None):
    st = load().fp4_gemm_mxfp4_grouped(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16),
                                       _ptr(row_offsets), E, total_M, N, K, _stream(stream))
    _check(st, "fp4_gemm_mxfp4_grouped")


def fp4_quant_dualscale(w_bf16, out_packed, out_fine, out_coarse, N, K, sf_layout=FP4_SF_SWIZZLED, stream=None):
    """bf16 weight -> DualScale codes, fine E8M0 scales and coarse float32 scales."""
    st = load().fp4_quant_dualscale(_ptr(w_bf16), _ptr(out_packed), _ptr(out_fine), _ptr(out_coarse), N, K,
                                    sf_layout, _stream(stream))
    _check(st, "fp4_quant_dualscale")


def fp4_gemm_mxfp4_dualscale(a, sa, b, sb, coarse, bias_bf16, out_bf16, M, N, K, workspace=None,
                             workspace_bytes=None, stream=None):
    """MXFP4 activations x DualScale weights (+ bias), bf16 out."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().fp4_gemm_mxfp4_dualscale(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(coarse), _ptr(bias_bf16),
                                         _ptr(out_bf16), M, N, K, _ptr(workspace), workspace_bytes, _stream(stream))
    _check(st, "fp4_gemm_mxfp4_dualscale")


# ----------------------------------------------------- around the FP4 linear


def fp4_fp8_act_scale_bytes(M, K):
    return load().fp4_fp8_act_scale_bytes(M, K)


def fp4_quant_act_fp8_b128(x_bf16, codes, scales, M, K, stream=None):
    """scales: float32 [ceil(K / 128)][M rounded up to 4]."""
    _check(load().fp4_quant_act_fp8_b128(_ptr(x_bf16), _ptr(codes), _ptr(scales), M, K, _stream(stream)),
           "fp4_quant_act_fp8_b128")


def fp4_quant_weight_fp8_b128(w_bf16, codes, scales, N, K, stream=None):
    """scales: float32 [ceil(N / 128)][ceil(K / 128)]."""
    _check(load().fp4_quant_weight_fp8_b128(_ptr(w_bf16), _ptr(codes), _ptr(scales), N, K, _stream(stream)),
           "fp4_quant_weight_fp8_b128")


def fp4_gemm_fp8_b128(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, stream=None):
    _check(load().fp4_gemm_fp8_b128(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                                    _stream(stream)), "fp4_gemm_fp8_b128")


def fp4_linear_fp8_b128_workspace_size(M, N, K):
    return load().fp4_linear_fp8_b128_workspace_size(M, N, K)


def fp4_linear_fp8_b128(x_bf16, b, sb, bias_bf16, out_bf16, M, N, K, workspace, workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().fp4_linear_fp8_b128(_ptr(x_bf16), _ptr(b), _ptr(sb), _ptr(bias_bf16), _ptr(out_bf16), M, N, K,
                                      _ptr(workspace), nbytes, _stream(stream)), "fp4_linear_fp8_b128")


_torch = None  # set with the first rope_params, kv_cache or table, which the calls on tensors need


def _need_torch():
    global _torch
    import torch as _torch


def _expect(t, dtype, count, what):
    """The kernels read these tensors by address alone: one of another type, with
    gaps, too short or on the host is refused here."""
    if t.dtype is not dtype or t.numel() < count or not t.is_contiguous() or not t.is_cuda:
        raise ValueError("%s: a contiguous device tensor of %s with at least %d elements" % (what, dtype, count))


class rope_params:
    """fp4_rope_params of a float32 table tensor [positions, rot_dim] (kept alive)."""

    def __init__(self, table, rot_dim, layout=FP4_ROPE_HALF, inverse=False):
        _need_torch()
        if table.dim() != 2 or table.shape[1] != rot_dim:
            raise ValueError("the table is [positions, rot_dim]")
        _expect(table, _torch.float32, 0, "table")
        self.table = table
        self.struct = fp4_rope_params(table.data_ptr(), table.shape[0], rot_dim, layout,
                                      FP4_ROPE_INVERSE if inverse else 0)
        self.ref = ctypes.byref(self.struct)


class kv_cache:
    """fp4_kv_cache of four tensors of one byte per element (kept alive): codes
    [pages, kv_heads, page_size, head_dim or head_dim / 2], scales [pages,
    kv_heads, page_size, head_dim / 32]."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, page_size, format):
        _need_torch()
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        for t in self.tensors:
            if not t.is_contiguous() or t.element_size() != 1 or not t.is_cuda:
                raise ValueError("cache tensors are contiguous bytes on the device")
        pages, heads, page, width = k_codes.shape
        dim = width if format == FP4_ACT_MXFP8 else 2 * width
        if page != page_size or v_codes.shape != k_codes.shape or any(
                s.shape != (pages, heads, page, dim // 32) for s in (k_scales, v_scales)):
            raise ValueError("cache tensors do not belong together")
        self.heads, self.dim = heads, dim
        self.struct = fp4_kv_cache(*(t.data_ptr() for t in self.tensors), pages, page_size, heads, dim, format)
        self.ref = ctypes.byref(self.struct)


def _pair(a, b, what):
    """The shape of two bf16 [tokens, heads, dim] tensors and their (token, head) strides."""
    shape = a.shape
    at, ah, ac = a.stride()
    bt, bh, bc = b.stride()
    kind = _torch.bfloat16
    if b.shape != shape or a.dtype is not kind or b.dtype is not kind or not a.is_cuda or not b.is_cuda or (
            (ac != 1 or bc != 1) and shape[2] != 1):
        raise ValueError("%s: bf16 device tensors [tokens, heads, dim] of one shape with contiguous heads" % what)
    return shape, at, ah, bt, bh


def _table_stride(t):
    """Rows and row stride of an int32 block table [batch, pages] (one row: its stride says nothing)."""
    rows, width = t.shape
    a, b = t.stride()
    if t.dtype is not _torch.int32 or (b != 1 and width != 1) or not t.is_cuda:
        raise ValueError("block_table: an int32 device tensor with contiguous rows")
    return rows, a if rows > 1 else width


def fp4_rope_table(table, positions, rot_dim, base, kind=FP4_ROPE_UNSCALED, factor=1.0, original_positions=0,
                   turns_fast=32.0, turns_slow=1.0, magnitude=1.0, stream=None):
    """Fills table float32 [positions, rot_dim] on the device."""
    if not isinstance(table, int):
        _need_torch()
        _expect(table, _torch.float32, positions * rot_dim, "table")
    sc = fp4_rope_scaling(kind, factor, original_positions, turns_fast, turns_slow, magnitude)
    _check(load().fp4_rope_table(_ptr(table), positions, rot_dim, base, ctypes.byref(sc), _stream(stream)),
           "fp4_rope_table")


def fp4_rope(x, out, positions, rope, stream=None):
    """x, out: bf16 [tokens, heads, head_dim] with any token and head strides
    that are multiples of 8; positions: int32 [tokens]; rope: rope_params."""
    (tokens, heads, dim), xt, xh, ot, oh = _pair(x, out, "x, out")
    _expect(positions, _torch.int32, tokens, "positions")
    _check(load().fp4_rope(x.data_ptr(), out.data_ptr(), positions.data_ptr(), rope.ref, tokens, heads, dim, xt, xh, ot,
                           oh, _stream(stream)), "fp4_rope")


def fp4_kv_append(cache, k, v, slots, rope=None, positions=None, stream=None):
    """k, v: bf16 [tokens, kv_heads, head_dim]; slots: int64 [tokens]; with
    `rope` the keys are rotated first (positions: int32 [tokens])."""
    (tokens, heads, dim), kt, kh, vt, vh = _pair(k, v, "k, v")
    if heads != cache.heads or dim != cache.dim:
        raise ValueError("k and v are [tokens, kv_heads, head_dim] of the cache")
    _expect(slots, _torch.int64, tokens, "slots")
    if rope is not None and positions is not None:
        _expect(positions, _torch.int32, tokens, "positions")
    _check(load().fp4_kv_append(cache.ref, k.data_ptr(), v.data_ptr(), tokens, kt, kh, vt, vh, slots.data_ptr(),
                                None if rope is None else rope.ref, _ptr(positions), _stream(stream)), "fp4_kv_append")


def fp4_kv_read(cache, block_table, cu_lens, k_out, v_out, stream=None):
    """block_table: int32 [batch, pages]; cu_lens: int32 [batch + 1]; k_out,
    v_out: contiguous bf16 [rows, kv_heads, head_dim]."""
    (rows, heads, dim), *_ = _pair(k_out, v_out, "k_out, v_out")
    if heads != cache.heads or dim != cache.dim or not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError("k_out and v_out are contiguous [rows, kv_heads, head_dim] of the cache")
    batch, stride = _table_stride(block_table)
    _expect(cu_lens, _torch.int32, batch + 1, "cu_lens")
    _check(load().fp4_kv_read(cache.ref, block_table.data_ptr(), stride, cu_lens.data_ptr(), batch, rows,
                              k_out.data_ptr(), v_out.data_ptr(), _stream(stream)), "fp4_kv_read")


def fp4_kv_attention_workspace_size(batch, tokens, q_heads, kv_heads, head_dim, max_seq_len, max_draft):
    return load().fp4_kv_attention_workspace_size(batch, tokens, q_heads, kv_heads, head_dim, max_seq_len, max_draft)


def fp4_kv_attention(cache, q, out, block_table, context_lens, q_offsets, max_seq_len, max_draft, workspace=None,
                     tree_mask=None, lse=None, softmax_scale=None, stream=None):
    """q, out: bf16 [tokens, q_heads, head_dim]; block_table: int32 [batch,
    pages]; context_lens: int32 [batch]; q_offsets: int32 [batch + 1];
    tree_mask: int32 or uint32 [tokens, words] or None (causal); lse: float32
    [tokens, q_heads] or None; softmax_scale defaults to head_dim ** -0.5."""
    (tokens, heads, dim), qt, qh, ot, oh = _pair(q, out, "q, out")
    if dim != cache.dim:
        raise ValueError("q and out are [tokens, q_heads, head_dim] with the cache's head_dim")
    batch, stride = _table_stride(block_table)
    _expect(context_lens, _torch.int32, batch, "context_lens")
    _expect(q_offsets, _torch.int32, batch + 1, "q_offsets")
    words = mask = log_sum = 0
    if tree_mask is not None:
        _, words = tree_mask.shape
        _expect(tree_mask, _torch.uint32 if tree_mask.dtype is _torch.uint32 else _torch.int32, tokens * words, "tree_mask")
        mask = tree_mask.data_ptr()
    if lse is not None:
        _expect(lse, _torch.float32, tokens * heads, "lse")
        log_sum = lse.data_ptr()
    if workspace is not None and not (workspace.is_contiguous() and workspace.is_cuda):
        raise ValueError("workspace: a contiguous device tensor")
    a = _attention_args(q.data_ptr(), out.data_ptr(), log_sum, qt, qh, ot, oh, block_table.data_ptr(), stride,
                        context_lens.data_ptr(), q_offsets.data_ptr(), mask, words, batch, tokens, heads, max_draft,
                        max_seq_len, dim ** -0.5 if softmax_scale is None else softmax_scale)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().fp4_kv_attention(cache.ref, a, _ptr(workspace), nbytes, _stream(stream)), "fp4_kv_attention")
