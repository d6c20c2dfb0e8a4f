"""Python binding of libtpgemm.so: the tile-primitive matrix multiply D = A.B + beta.C.

Argument marshalling only. Every step of the computation runs in the CUDA
kernels of ``libtpgemm.so``; this module turns torch tensors (or raw integer
device pointers) and streams into the C-ABI call declared in
``include/tpgemm.h``. The functions keep the C names; ``gemm`` is a
convenience wrapper that allocates D with torch when no output is given.

There is no fallback: if the library has not been built, every call raises.
Build it with ``tile_primitive_tensor_gb300.build.build()``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading
import typing

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtpgemm.so")
# Debug build (device-side bounds checks; built on request by build(debug=True)).
LIB_PATH_DEBUG = os.path.join(_HERE, "_lib", "libtpgemm_debug.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "tpgemm.h")

# tpgemm_dtype
TPGEMM_F16 = 0
TPGEMM_BF16 = 1
TPGEMM_E4M3 = 2
TPGEMM_E5M2 = 3
TPGEMM_E2M1 = 4  # fp4, packed two per byte (element 2i in the low nibble of byte i)
# tpgemm_status
TPGEMM_OK = 0
TPGEMM_ERR_SHAPE = 1
TPGEMM_ERR_DTYPE = 2
TPGEMM_ERR_BETA = 3
TPGEMM_ERR_NULL = 4
TPGEMM_ERR_ALIGN = 5
TPGEMM_ERR_ALIAS = 6
TPGEMM_ERR_ARCH = 7
TPGEMM_ERR_LAUNCH = 8
TPGEMM_ERR_TIMEOUT = 9
TPGEMM_ERR_PATH = 10
TPGEMM_ERR_BOUNDS = 11
# tpgemm_path
TPGEMM_PATH_AUTO = 0
TPGEMM_PATH_TCGEN05 = 1
TPGEMM_PATH_MMA_SYNC = 2
# tpgemm_cp_swizzle
TPGEMM_CP_SWIZZLE_NONE = 0
TPGEMM_CP_SWIZZLE_32B = 1
TPGEMM_CP_SWIZZLE_64B = 2
TPGEMM_CP_SWIZZLE_128B = 3
# tpgemm_cp_shape
TPGEMM_CP_AUTO = 0
TPGEMM_CP_128x256b = 1
TPGEMM_CP_4x256b = 2
TPGEMM_CP_128x128b = 3
TPGEMM_CP_64x128b_WARPX2_02_13 = 4
TPGEMM_CP_64x128b_WARPX2_01_23 = 5
TPGEMM_CP_32x128b_WARPX4 = 6
# tpgemm_tmem_shape
TPGEMM_TMEM_32x32b = 0
TPGEMM_TMEM_16x64b = 1
TPGEMM_TMEM_16x128b = 2
TPGEMM_TMEM_16x256b = 3
# tpgemm_cp_lanes
TPGEMM_CP_LANES_ROWS = 0
TPGEMM_CP_LANES_QUADRANTS = 1
TPGEMM_CP_LANES_PAIRS_02_13 = 2
TPGEMM_CP_LANES_PAIRS_01_23 = 3
TPGEMM_CP_LANES_ALL_QUADS = 4


# tpgemm_elem (the first four codes are tpgemm_dtype's)
TPGEMM_ELEM_F16 = 0
TPGEMM_ELEM_BF16 = 1
TPGEMM_ELEM_E4M3 = 2
TPGEMM_ELEM_E5M2 = 3
TPGEMM_ELEM_F32 = 8
# tpgemm_act
TPGEMM_ACT_NONE = 0
TPGEMM_ACT_RELU = 1
TPGEMM_ACT_SILU = 2
TPGEMM_ACT_GELU = 3
TPGEMM_ACT_GELU_TANH = 4
# tpgemm_scale_mode
TPGEMM_SCALE_NONE = 0
TPGEMM_SCALE_ROW = 1
TPGEMM_SCALE_MX = 2


class LinearDesc(ctypes.Structure):
    """tpgemm_linear_desc: sizes, row strides, types and activation of a linear layer."""
    _fields_ = [(n, ctypes.c_int64) for n in ("M", "N", "K", "lda", "ldw", "ldr", "ldy", "ldz")] + \
        [(n, ctypes.c_int) for n in ("dtype", "out", "act")]


class LinearGradDesc(ctypes.Structure):
    """tpgemm_linear_grad_desc: as LinearDesc, for the gradients."""
    _fields_ = [(n, ctypes.c_int64)
                for n in ("M", "N", "K", "lddy", "ldz", "lda", "ldw", "ldda", "lddw")] + \
        [(n, ctypes.c_int) for n in ("dtype", "grad", "act")]


class RmsNormDesc(ctypes.Structure):
    """tpgemm_rmsnorm_desc: sizes, row strides, types, scale mode and eps of a norm."""
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "ldx", "ldr", "ldh", "ldy")] + \
        [(n, ctypes.c_int) for n in ("x", "gamma", "y", "scale")] + [("eps", ctypes.c_float)]


class RmsNormGradDesc(ctypes.Structure):
    """tpgemm_rmsnorm_grad_desc: as RmsNormDesc, for the gradients."""
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "lddy", "ldh", "lddh", "lddx")] + \
        [(n, ctypes.c_int) for n in ("x", "gamma", "grad")]


# tpgemm_drop: probability, seed, offset and the device address of a counter (or None). (Its
# members stand in the descriptions themselves: a structure of its own costs half a microsecond.)
_DROP = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
         ("counter", ctypes.c_void_p)]


class DropoutDesc(ctypes.Structure):
    """tpgemm_dropout_desc: sizes, row strides, type and random numbers of a dropout."""
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "ldx", "ldr", "ldy")] + \
        [("x", ctypes.c_int)] + _DROP


class LayerNormDesc(ctypes.Structure):
    """tpgemm_layernorm_desc: as RmsNormDesc, and the dropout before the norm."""
    _fields_ = RmsNormDesc._fields_ + _DROP


class LayerNormGradDesc(ctypes.Structure):
    """tpgemm_layernorm_grad_desc: as LayerNormDesc, for the gradients."""
    _fields_ = [(n, ctypes.c_int64)
                for n in ("rows", "cols", "lddy", "ldh", "lddh", "lddx", "lddr")] + \
        [(n, ctypes.c_int) for n in ("x", "gamma", "grad")] + _DROP


class CpDesc(ctypes.Structure):
    """tpgemm_cp_desc: a shared-memory region and where its rows go in tensor memory."""
    _fields_ = [("rows", ctypes.c_int), ("row_bits", ctypes.c_int), ("swizzle", ctypes.c_int),
                ("lbo_bytes", ctypes.c_uint32), ("sbo_bytes", ctypes.c_uint32),
                ("smem_offset", ctypes.c_uint32), ("tmem_col", ctypes.c_int),
                ("lane_offset", ctypes.c_int), ("lanes", ctypes.c_int), ("shape", ctypes.c_int),
                ("cta_group", ctypes.c_int)]


class TpgemmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.detail = detail
        super().__init__(f"tpgemm status {status} ({tpgemm_status_string(status)}): {detail}")


_lib = None
_lock = threading.Lock()


def _open(path):
    """A ctypes handle of a libtpgemm build with every declared signature set."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run tile_primitive_tensor_gb300.build.build() "
            "(nvcc for sm_103a). There is no CPU fallback.")
    lib = ctypes.CDLL(path)
    vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    gemm_args = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, cf, vp]
    lib.tpgemm_gemm.argtypes = gemm_args
    lib.tpgemm_gemm.restype = ci
    lib.tpgemm_gemm_path.argtypes = gemm_args + [ci]
    lib.tpgemm_gemm_path.restype = ci
    lib.tpgemm_gemm_noalloc.argtypes = gemm_args
    lib.tpgemm_gemm_noalloc.restype = ci
    lib.tpgemm_test_gemm_withhold_fill.argtypes = gemm_args
    lib.tpgemm_test_gemm_withhold_fill.restype = ci
    lib.tpgemm_reload_tuning.argtypes = []
    lib.tpgemm_reload_tuning.restype = None
    lib.tpgemm_gemm_host.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, cf, vp,
                                     ctypes.c_size_t, vp]
    lib.tpgemm_gemm_host.restype = ci
    lib.tpgemm_gemm_host_workspace_bytes.argtypes = [i64, i64, i64, ci, cf]
    lib.tpgemm_gemm_host_workspace_bytes.restype = ctypes.c_size_t
    lib.tpgemm_status_string.argtypes = [ci]
    lib.tpgemm_status_string.restype = ctypes.c_char_p
    lib.tpgemm_last_error_detail.argtypes = []
    lib.tpgemm_last_error_detail.restype = ctypes.c_char_p
    lib.tpgemm_last_device_error.argtypes = []
    lib.tpgemm_last_device_error.restype = ci
    lib.tpgemm_describe_plan.argtypes = [i64, i64, i64, ci, ci, ci, cf, ci, ctypes.c_char_p, ci]
    lib.tpgemm_describe_plan.restype = ci
    lib.tpgemm_last_plan.argtypes = [ctypes.c_char_p, ci]
    lib.tpgemm_last_plan.restype = ci
    u32 = ctypes.c_uint32
    lib.tpgemm_encode_smem_desc.argtypes = [u32, u32, u32, ci]
    lib.tpgemm_encode_smem_desc.restype = ctypes.c_uint64
    lib.tpgemm_encode_idesc.argtypes = [ci, ci, ci, ci, ci]
    lib.tpgemm_encode_idesc.restype = u32
    lib.tpgemm_encode_idesc_mx.argtypes = [ci, ci, ci, ci, ci]
    lib.tpgemm_encode_idesc_mx.restype = u32
    sz = ctypes.c_size_t
    lib.tpgemm_gemm_mx.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, cf, vp, sz, vp]
    lib.tpgemm_gemm_mx.restype = ci
    lib.tpgemm_gemm_mx_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tpgemm_gemm_mx_workspace_bytes.restype = sz
    lib.tpgemm_linear.argtypes = [vp] * 8 + [ctypes.POINTER(LinearDesc), vp, sz, vp]
    lib.tpgemm_linear.restype = ci
    lib.tpgemm_linear_workspace_bytes.argtypes = [vp, vp, ctypes.POINTER(LinearDesc)]
    lib.tpgemm_linear_workspace_bytes.restype = sz
    lib.tpgemm_linear_backward.argtypes = [vp] * 7 + [ctypes.POINTER(LinearGradDesc), vp, sz, vp]
    lib.tpgemm_linear_backward.restype = ci
    lib.tpgemm_linear_backward_workspace_bytes.argtypes = [vp, vp, vp,
                                                           ctypes.POINTER(LinearGradDesc)]
    lib.tpgemm_linear_backward_workspace_bytes.restype = sz
    lib.tpgemm_gated_linear.argtypes = [vp] * 7 + [ctypes.POINTER(LinearDesc), vp, sz, vp]
    lib.tpgemm_gated_linear.restype = ci
    lib.tpgemm_gated_linear_workspace_bytes.argtypes = [vp, vp, ctypes.POINTER(LinearDesc)]
    lib.tpgemm_gated_linear_workspace_bytes.restype = sz
    lib.tpgemm_gated_linear_backward.argtypes = [vp] * 7 + [ctypes.POINTER(LinearGradDesc), vp, sz, vp]
    lib.tpgemm_gated_linear_backward.restype = ci
    lib.tpgemm_gated_linear_backward_workspace_bytes.argtypes = [vp, vp, vp,
                                                                 ctypes.POINTER(LinearGradDesc)]
    lib.tpgemm_gated_linear_backward_workspace_bytes.restype = sz
    lib.tpgemm_rmsnorm.argtypes = [vp] * 7 + [ctypes.POINTER(RmsNormDesc), vp]
    lib.tpgemm_rmsnorm.restype = ci
    lib.tpgemm_rmsnorm_backward.argtypes = [vp] * 7 + [ctypes.POINTER(RmsNormGradDesc), vp, sz, vp]
    lib.tpgemm_rmsnorm_backward.restype = ci
    lib.tpgemm_rmsnorm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.tpgemm_rmsnorm_backward_workspace_bytes.restype = sz
    lib.tpgemm_dropout.argtypes = [vp] * 3 + [ctypes.POINTER(DropoutDesc), vp]
    lib.tpgemm_dropout.restype = ci
    lib.tpgemm_layernorm.argtypes = [vp] * 9 + [ctypes.POINTER(LayerNormDesc), vp]
    lib.tpgemm_layernorm.restype = ci
    lib.tpgemm_layernorm_backward.argtypes = [vp] * 10 + [ctypes.POINTER(LayerNormGradDesc), vp, sz, vp]
    lib.tpgemm_layernorm_backward.restype = ci
    lib.tpgemm_layernorm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.tpgemm_layernorm_backward_workspace_bytes.restype = sz
    lib.tpgemm_version.argtypes = []
    lib.tpgemm_version.restype = ctypes.c_char_p
    lib.tpgemm_cp_parse_shape.argtypes = [ctypes.c_char_p, ctypes.POINTER(ci)]
    lib.tpgemm_cp_parse_shape.restype = ci
    lib.tpgemm_cp_plan.argtypes = [ctypes.POINTER(CpDesc), ctypes.c_char_p, ci]
    lib.tpgemm_cp_plan.restype = ci
    lib.tpgemm_cp_roundtrip.argtypes = [vp, vp, ctypes.c_size_t, ctypes.POINTER(CpDesc),
                                        ctypes.c_uint32, ci, vp]
    lib.tpgemm_cp_roundtrip.restype = ci
    lib.tpgemm_cp_roundtrip_repeat.argtypes = [vp, vp, ctypes.c_size_t, ctypes.POINTER(CpDesc),
                                               ctypes.c_uint32, ci, ci, ci, ci, vp]
    lib.tpgemm_cp_roundtrip_repeat.restype = ci
    lib.tpgemm_tmem_ldst_roundtrip.argtypes = [vp, vp, vp, ci, ci, ci, ci, ctypes.c_uint32,
                                               vp]
    lib.tpgemm_tmem_ldst_roundtrip.restype = ci
    lib.tpgemm_vcopy_plan.argtypes = [ctypes.POINTER(VcopyDesc), ctypes.c_char_p, ci]
    lib.tpgemm_vcopy_plan.restype = ci
    lib.tpgemm_vcopy_roundtrip.argtypes = [vp, vp, ctypes.c_size_t, ctypes.POINTER(VcopyDesc),
                                           ci, i64, vp, vp]
    lib.tpgemm_vcopy_roundtrip.restype = ci
    return lib


_lib_debug = None


def _load():
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(LIB_PATH)
        return _lib


def debug_library():
    """The ctypes handle of libtpgemm_debug.so (same C ABI, device-side bounds
    checks that report TPGEMM_ERR_BOUNDS); build it with build(debug=True)."""
    global _lib_debug
    with _lock:
        if _lib_debug is None:
            _lib_debug = _open(LIB_PATH_DEBUG)
        return _lib_debug


def library():
    """The loaded ctypes handle of libtpgemm.so."""
    return _load()


def header_functions():
    """Names of the functions declared in include/tpgemm.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tpgemm_\w+)\s*\(", text)))


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    raise TypeError(f"expected a tensor or an integer device pointer, got {type(x)!r}")


def _stream(s) -> int | None:
    if s is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    raise TypeError(f"expected a torch.cuda.Stream, an integer cudaStream_t or None, got {type(s)!r}")


def tpgemm_gemm(D, A, B, C, M, N, K, transA, transB, dtype, beta, stream=None) -> int:
    """Enqueue D = A.B + beta.C; returns the tpgemm_status code."""
    return int(_load().tpgemm_gemm(_ptr(D), _ptr(A), _ptr(B), _ptr(C), int(M), int(N), int(K),
                                   int(bool(transA)), int(bool(transB)), int(dtype), float(beta),
                                   _stream(stream)))


def tpgemm_gemm_path(D, A, B, C, M, N, K, transA, transB, dtype, beta, stream=None,
                     path=TPGEMM_PATH_AUTO) -> int:
    return int(_load().tpgemm_gemm_path(_ptr(D), _ptr(A), _ptr(B), _ptr(C), int(M), int(N),
                                        int(K), int(bool(transA)), int(bool(transB)), int(dtype),
                                        float(beta), _stream(stream), int(path)))


def tpgemm_gemm_noalloc(D, A, B, C, M, N, K, transA, transB, dtype, beta, stream=None) -> int:
    """tpgemm_gemm that allocates no device memory (static stream-K scratch)."""
    return int(_load().tpgemm_gemm_noalloc(_ptr(D), _ptr(A), _ptr(B), _ptr(C), int(M), int(N),
                                           int(K), int(bool(transA)), int(bool(transB)),
                                           int(dtype), float(beta), _stream(stream)))


def tpgemm_gemm_mx(D, A, B, C, SFA, SFB, M, N, K, dtype, beta, workspace, workspace_bytes,
                   stream=None) -> int:
    """Enqueue the block-scaled fp8 multiply (A [M,K], B [N,K], E8M0 scales
    SFA [M, ceil(K/32)], SFB [N, ceil(K/32)]); returns the tpgemm_status code."""
    return int(_load().tpgemm_gemm_mx(_ptr(D), _ptr(A), _ptr(B), _ptr(C), _ptr(SFA), _ptr(SFB),
                                      int(M), int(N), int(K), int(dtype), float(beta),
                                      _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tpgemm_gemm_mx_workspace_bytes(M, N, K) -> int:
    return int(_load().tpgemm_gemm_mx_workspace_bytes(int(M), int(N), int(K)))


def tpgemm_encode_idesc_mx(dtype, m, n, a_sf_id, b_sf_id) -> int:
    return int(_load().tpgemm_encode_idesc_mx(int(dtype), int(m), int(n), int(a_sf_id),
                                              int(b_sf_id)))


def tpgemm_test_gemm_withhold_fill(D, A, B, C, M, N, K, transA, transB, dtype, beta,
                                   stream=None) -> int:
    """Test aid: the tcgen05 GEMM with CTA 0's first stage fill withheld."""
    return int(_load().tpgemm_test_gemm_withhold_fill(
        _ptr(D), _ptr(A), _ptr(B), _ptr(C), int(M), int(N), int(K), int(bool(transA)),
        int(bool(transB)), int(dtype), float(beta), _stream(stream)))


def tpgemm_reload_tuning() -> None:
    """Re-read the TPGEMM_* planner overrides from the environment."""
    _load().tpgemm_reload_tuning()


def tpgemm_gemm_host_workspace_bytes(M, N, K, dtype, beta) -> int:
    return int(_load().tpgemm_gemm_host_workspace_bytes(int(M), int(N), int(K), int(dtype),
                                                        float(beta)))


def tpgemm_gemm_host(D_host, A_host, B_host, C_host, M, N, K, transA, transB, dtype, beta,
                     workspace, workspace_bytes, stream=None) -> int:
    """Enqueue D = A.B + beta.C on host buffers (copies pipelined with the multiply)."""
    return int(_load().tpgemm_gemm_host(_ptr(D_host), _ptr(A_host), _ptr(B_host), _ptr(C_host),
                                        int(M), int(N), int(K), int(bool(transA)),
                                        int(bool(transB)), int(dtype), float(beta),
                                        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tpgemm_status_string(status: int) -> str:
    return _load().tpgemm_status_string(int(status)).decode()


def tpgemm_last_error_detail() -> str:
    return _load().tpgemm_last_error_detail().decode()


def tpgemm_last_device_error() -> int:
    return int(_load().tpgemm_last_device_error())


def tpgemm_describe_plan(M, N, K, transA, transB, dtype, beta, path=TPGEMM_PATH_AUTO):
    buf = ctypes.create_string_buffer(640)
    st = int(_load().tpgemm_describe_plan(int(M), int(N), int(K), int(bool(transA)),
                                          int(bool(transB)), int(dtype), float(beta), int(path),
                                          buf, 640))
    return st, buf.value.decode()


def tpgemm_encode_smem_desc(start_addr, lbo_bytes, sbo_bytes, swizzle) -> int:
    return int(_load().tpgemm_encode_smem_desc(int(start_addr), int(lbo_bytes), int(sbo_bytes),
                                               int(swizzle)))


def tpgemm_encode_idesc(dtype, a_mn_major, b_mn_major, m, n) -> int:
    return int(_load().tpgemm_encode_idesc(int(dtype), int(bool(a_mn_major)),
                                           int(bool(b_mn_major)), int(m), int(n)))


def tpgemm_last_plan():
    buf = ctypes.create_string_buffer(640)
    st = int(_load().tpgemm_last_plan(buf, 640))
    return st, buf.value.decode()


class VcopyDesc(ctypes.Structure):
    """tpgemm_vcopy_desc: a global region, its shared placement and the copying scope."""
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("elem_bytes", ctypes.c_int),
                ("g_row_stride", ctypes.c_int64), ("g_offset", ctypes.c_int64),
                ("s_row_stride", ctypes.c_int), ("s_offset", ctypes.c_int),
                ("s_swizzle", ctypes.c_int), ("threads", ctypes.c_int)]


def vcopy_desc(rows, cols, elem_bytes, *, g_row_stride=None, g_offset=0, s_row_stride=None,
               s_offset=0, s_swizzle=0, threads=32) -> VcopyDesc:
    return VcopyDesc(int(rows), int(cols), int(elem_bytes),
                     int(cols if g_row_stride is None else g_row_stride), int(g_offset),
                     int(cols if s_row_stride is None else s_row_stride), int(s_offset),
                     int(s_swizzle), int(threads))


def tpgemm_vcopy_plan(desc: VcopyDesc):
    buf = ctypes.create_string_buffer(512)
    st = int(_load().tpgemm_vcopy_plan(ctypes.byref(desc), buf, 512))
    return st, buf.value.decode()


def tpgemm_vcopy_roundtrip(dst, src, buffer_bytes, desc: VcopyDesc, ctas=1, cta_stride=0,
                           smem_out=None, stream=None) -> int:
    return int(_load().tpgemm_vcopy_roundtrip(_ptr(dst), _ptr(src), int(buffer_bytes),
                                              ctypes.byref(desc), int(ctas), int(cta_stride),
                                              _ptr(smem_out), _stream(stream)))


def cp_desc(rows, row_bits, *, swizzle=TPGEMM_CP_SWIZZLE_NONE, lbo=0, sbo=0, smem_offset=0,
            tmem_col=0, lane_offset=0, lanes=TPGEMM_CP_LANES_ROWS, shape=TPGEMM_CP_AUTO,
            cta_group=1) -> CpDesc:
    return CpDesc(int(rows), int(row_bits), int(swizzle), int(lbo), int(sbo), int(smem_offset),
                  int(tmem_col), int(lane_offset), int(lanes), int(shape), int(cta_group))


def tpgemm_cp_parse_shape(name: str):
    """(status, tpgemm_cp_shape) for a form name such as "64x128b.warpx2::02_13"."""
    out = ctypes.c_int(0)
    st = int(_load().tpgemm_cp_parse_shape(name.encode(), ctypes.byref(out)))
    return st, out.value


def tpgemm_cp_plan(desc: CpDesc):
    """(status, text): the planned tcgen05.cp instructions, or the rejection reason."""
    buf = ctypes.create_string_buffer(16384)
    st = int(_load().tpgemm_cp_plan(ctypes.byref(desc), buf, 16384))
    return st, buf.value.decode()


def tpgemm_cp_roundtrip(tmem_out, smem_image, image_bytes, desc: CpDesc, fill_base, ncols,
                        stream=None) -> int:
    """Enqueue image -> shared memory -> tcgen05.cp -> tensor memory -> tmem_out."""
    return int(_load().tpgemm_cp_roundtrip(_ptr(tmem_out), _ptr(smem_image), int(image_bytes),
                                           ctypes.byref(desc), int(fill_base) & 0xFFFFFFFF,
                                           int(ncols), _stream(stream)))


def tpgemm_cp_roundtrip_repeat(tmem_out, smem_image, image_bytes, desc: CpDesc, fill_base, ncols,
                               repeat, ctas, issuers=1, stream=None) -> int:
    """The round trip on `ctas` CTAs, each issuing the planned copy `repeat` times from
    `issuers` threads."""
    return int(_load().tpgemm_cp_roundtrip_repeat(_ptr(tmem_out), _ptr(smem_image),
                                                  int(image_bytes), ctypes.byref(desc),
                                                  int(fill_base) & 0xFFFFFFFF, int(ncols),
                                                  int(repeat), int(ctas), int(issuers),
                                                  _stream(stream)))


def tpgemm_tmem_ldst_roundtrip(regs_out, tmem_out, regs_in, st_shape, ld_shape, cols, tmem_col,
                               fill_base, stream=None) -> int:
    """Registers -> tensor memory (st_shape) -> .32x32b read-back and ld_shape load."""
    return int(_load().tpgemm_tmem_ldst_roundtrip(_ptr(regs_out), _ptr(tmem_out), _ptr(regs_in),
                                                  int(st_shape), int(ld_shape), int(cols),
                                                  int(tmem_col), int(fill_base) & 0xFFFFFFFF,
                                                  _stream(stream)))


def tpgemm_version() -> str:
    return _load().tpgemm_version().decode()


def check(status: int) -> None:
    if status != TPGEMM_OK:
        raise TpgemmError(status, tpgemm_last_error_detail())


def dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.float16:
        return TPGEMM_F16
    if torch_dtype == torch.bfloat16:
        return TPGEMM_BF16
    if torch_dtype == torch.float8_e4m3fn:
        return TPGEMM_E4M3
    if torch_dtype == torch.float8_e5m2:
        return TPGEMM_E5M2
    raise TypeError(f"A and B must be float16, bfloat16, float8_e4m3fn or float8_e5m2, "
                    f"got {torch_dtype}")


def gemm_mx(A, B, SFA, SFB, C=None, *, beta=None, out=None, workspace=None, stream=None,
            dtype=None):
    """Block-scaled fp8 / fp4 D = (A.SA)(B.SB)^T + beta.C on CUDA tensors.

    A is fp8 [M, K], B fp8 [N, K] (same dtype), or both fp4 as uint8 [M, K/2]
    and [N, K/2] (two codes per byte) with dtype=TPGEMM_E2M1; SFA uint8
    [M, ceil(K/32)] and SFB uint8 [N, ceil(K/32)] E8M0 scales, C float32 [M, N].
    The scale-packing workspace is allocated here with torch unless given.
    stream (by default the current one) is current for the call: its memory
    holds the output and the workspace."""
    if stream is not None:
        with _current(stream, A):
            return gemm_mx(A, B, SFA, SFB, C, beta=beta, out=out, workspace=workspace, dtype=dtype)
    import torch
    if beta is None:
        beta = 0.0 if C is None else 1.0
    M, K = A.shape
    N = B.shape[0]
    if dtype == TPGEMM_E2M1:
        K *= 2
    code = dtype if dtype is not None else dtype_code(A.dtype)
    if B.shape[1] != A.shape[1] or A.dtype != B.dtype:
        raise ValueError("A must be [M, K] and B [N, K] of the same fp8 / fp4 dtype")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    wsb = tpgemm_gemm_mx_workspace_bytes(M, N, K)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=A.device)
    check(tpgemm_gemm_mx(out, A, B, C, SFA, SFB, M, N, K, code, beta, workspace,
                         workspace.numel() * workspace.element_size()))
    return out


def gemm(A, B, C=None, *, beta=None, transA=False, transB=False, out=None, stream=None,
         path=TPGEMM_PATH_AUTO):
    """D = A.B + beta.C on CUDA tensors; returns D (float32 [M, N]).

    A is [M, K] (or [K, M] with transA), B is [K, N] (or [N, K] with transB),
    C is float32 [M, N]. beta defaults to 1 when C is given, else 0. ``out``
    may be C itself for the in-place form D += A.B. stream (by default the
    current one) is current for the call: its memory holds the output.
    """
    if stream is not None:
        with _current(stream, A):
            return gemm(A, B, C, beta=beta, transA=transA, transB=transB, out=out, path=path)
    import torch
    if beta is None:
        beta = 0.0 if C is None else 1.0
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = (A.shape[1], A.shape[0]) if transA else (A.shape[0], A.shape[1])
    Kb, N = (B.shape[1], B.shape[0]) if transB else (B.shape[0], B.shape[1])
    if K != Kb:
        raise ValueError(f"inner dimensions differ: A gives K={K}, B gives K={Kb}")
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same dtype")
    for name, t in (("A", A), ("B", B), ("C", C), ("out", out)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (dense row-major)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    check(tpgemm_gemm_path(out, A, B, C if beta else C, M, N, K, transA, transB,
                           dtype_code(A.dtype), beta, None, path))
    return out


# ------------------------------------------------ the operators around the multiply
def tpgemm_linear(Y, Z, A, W, scale_a, scale_w, bias, R, desc: LinearDesc, workspace=None,
                  workspace_bytes=0, stream=None) -> int:
    """Enqueue Y = act(scale_a scale_w A.W^T + bias) + R; returns the tpgemm_status code."""
    return int(_load().tpgemm_linear(_ptr(Y), _ptr(Z), _ptr(A), _ptr(W), _ptr(scale_a),
                                     _ptr(scale_w), _ptr(bias), _ptr(R), ctypes.byref(desc),
                                     _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tpgemm_linear_workspace_bytes(A, W, desc: LinearDesc) -> int:
    return int(_load().tpgemm_linear_workspace_bytes(_ptr(A), _ptr(W), ctypes.byref(desc)))


def tpgemm_linear_backward(dA, dW, dbias, dY, A, W, Z, desc: LinearGradDesc, workspace=None,
                           workspace_bytes=0, stream=None) -> int:
    """Enqueue the gradients of a linear layer; returns the tpgemm_status code."""
    return int(_load().tpgemm_linear_backward(_ptr(dA), _ptr(dW), _ptr(dbias), _ptr(dY), _ptr(A),
                                              _ptr(W), _ptr(Z), ctypes.byref(desc),
                                              _ptr(workspace), int(workspace_bytes),
                                              _stream(stream)))


def tpgemm_linear_backward_workspace_bytes(dY, A, W, desc: LinearGradDesc) -> int:
    return int(_load().tpgemm_linear_backward_workspace_bytes(_ptr(dY), _ptr(A), _ptr(W),
                                                              ctypes.byref(desc)))


def tpgemm_gated_linear(Y, Z, A, W, scale_a, scale_w, bias, desc: LinearDesc, workspace=None,
                        workspace_bytes=0, stream=None) -> int:
    """Enqueue a gated linear layer; returns the tpgemm_status code."""
    return int(_load().tpgemm_gated_linear(_ptr(Y), _ptr(Z), _ptr(A), _ptr(W), _ptr(scale_a),
                                           _ptr(scale_w), _ptr(bias), ctypes.byref(desc),
                                           _ptr(workspace), int(workspace_bytes),
                                           _stream(stream)))


def tpgemm_gated_linear_workspace_bytes(A, W, desc: LinearDesc) -> int:
    return int(_load().tpgemm_gated_linear_workspace_bytes(_ptr(A), _ptr(W), ctypes.byref(desc)))


def tpgemm_gated_linear_backward(dA, dW, dbias, dY, A, W, Z, desc: LinearGradDesc, workspace=None,
                                 workspace_bytes=0, stream=None) -> int:
    """Enqueue the gradients of a gated linear layer; returns the tpgemm_status code."""
    return int(_load().tpgemm_gated_linear_backward(
        _ptr(dA), _ptr(dW), _ptr(dbias), _ptr(dY), _ptr(A), _ptr(W), _ptr(Z), ctypes.byref(desc),
        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tpgemm_gated_linear_backward_workspace_bytes(dY, A, W, desc: LinearGradDesc) -> int:
    return int(_load().tpgemm_gated_linear_backward_workspace_bytes(_ptr(dY), _ptr(A), _ptr(W),
                                                                    ctypes.byref(desc)))


def tpgemm_rmsnorm(Y, H, scale, rstd, X, R, gamma, desc: RmsNormDesc, stream=None) -> int:
    """Enqueue a root-mean-square norm; returns the tpgemm_status code."""
    return int(_load().tpgemm_rmsnorm(_ptr(Y), _ptr(H), _ptr(scale), _ptr(rstd), _ptr(X), _ptr(R),
                                      _ptr(gamma), ctypes.byref(desc), _stream(stream)))


def tpgemm_rmsnorm_backward(dX, dgamma, dY, H, rstd, gamma, dH, desc: RmsNormGradDesc,
                            workspace=None, workspace_bytes=0, stream=None) -> int:
    """Enqueue the gradients of a root-mean-square norm; returns the tpgemm_status code."""
    return int(_load().tpgemm_rmsnorm_backward(_ptr(dX), _ptr(dgamma), _ptr(dY), _ptr(H),
                                               _ptr(rstd), _ptr(gamma), _ptr(dH),
                                               ctypes.byref(desc), _ptr(workspace),
                                               int(workspace_bytes), _stream(stream)))


def tpgemm_rmsnorm_backward_workspace_bytes(rows, cols) -> int:
    return int(_load().tpgemm_rmsnorm_backward_workspace_bytes(int(rows), int(cols)))


def tpgemm_dropout(Y, X, R, desc: DropoutDesc, stream=None) -> int:
    """Enqueue Y = drop(X) + R; returns the tpgemm_status code."""
    return int(_load().tpgemm_dropout(_ptr(Y), _ptr(X), _ptr(R), ctypes.byref(desc),
                                      _stream(stream)))


def tpgemm_layernorm(Y, H, scale, mean, rstd, X, R, gamma, beta, desc: LayerNormDesc,
                     stream=None) -> int:
    """Enqueue a layer norm; returns the tpgemm_status code."""
    return int(_load().tpgemm_layernorm(_ptr(Y), _ptr(H), _ptr(scale), _ptr(mean), _ptr(rstd),
                                        _ptr(X), _ptr(R), _ptr(gamma), _ptr(beta),
                                        ctypes.byref(desc), _stream(stream)))


def tpgemm_layernorm_backward(dX, dR, dgamma, dbeta, dY, H, mean, rstd, gamma, dH,
                              desc: LayerNormGradDesc, workspace=None, workspace_bytes=0,
                              stream=None) -> int:
    """Enqueue the gradients of a layer norm; returns the tpgemm_status code."""
    return int(_load().tpgemm_layernorm_backward(_ptr(dX), _ptr(dR), _ptr(dgamma), _ptr(dbeta),
                                                 _ptr(dY), _ptr(H), _ptr(mean), _ptr(rstd),
                                                 _ptr(gamma), _ptr(dH), ctypes.byref(desc),
                                                 _ptr(workspace), int(workspace_bytes),
                                                 _stream(stream)))


def tpgemm_layernorm_backward_workspace_bytes(rows, cols) -> int:
    return int(_load().tpgemm_layernorm_backward_workspace_bytes(int(rows), int(cols)))


_ACTS = {"none": TPGEMM_ACT_NONE, "relu": TPGEMM_ACT_RELU, "silu": TPGEMM_ACT_SILU,
         "gelu": TPGEMM_ACT_GELU, "gelu_tanh": TPGEMM_ACT_GELU_TANH}
_SCALES = {None: TPGEMM_SCALE_NONE, "row": TPGEMM_SCALE_ROW, "mx": TPGEMM_SCALE_MX}
_ELEMS = {}


def elem_code(torch_dtype) -> int:
    """The tpgemm_elem code of a torch dtype."""
    if not _ELEMS:
        import torch
        _ELEMS.update({torch.float16: TPGEMM_ELEM_F16, torch.bfloat16: TPGEMM_ELEM_BF16,
                       torch.float8_e4m3fn: TPGEMM_ELEM_E4M3, torch.float8_e5m2: TPGEMM_ELEM_E5M2,
                       torch.float32: TPGEMM_ELEM_F32})
    code = _ELEMS.get(torch_dtype)
    if code is None:
        raise TypeError(f"unsupported element type {torch_dtype}")
    return code


def _act_code(act) -> int:
    if act in _ACTS:
        return _ACTS[act]
    raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")


def _matrix(name, t, rows, cols, dtype, index) -> int:
    """Checks a [rows, cols] argument of unit column stride; returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not cuda:{index}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride, got {s1}")
    if rows <= 1 or cols == 0:
        return cols
    if s0 < cols:
        raise ValueError(f"{name}: row stride {s0} is less than its {cols} columns")
    return s0


def _vector(name, t, n, dtype, index) -> int:
    """Checks a dense vector argument; returns its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not cuda:{index}")
    if t.shape != (n,) or (n > 1 and t.stride()[0] != 1):
        raise ValueError(f"{name} must be a dense vector of {n}")
    return t.data_ptr()


_torch = None


def _import_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _sizes(name, t):
    """Rows, columns, device index and device of the 2-D CUDA tensor that leads a call."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return shape[0], shape[1], index, t.device


def _current(stream, t):
    """A context in which `stream` (a torch.cuda.Stream or an integer cudaStream_t of the CUDA
    tensor t's device) is torch's current stream. A call on a given stream runs in it whole, so
    that its outputs too come from that stream's memory: taken from the stream current before,
    they could be blocks that work there still reads, or go back to it while this stream writes."""
    torch = _torch or _import_torch()
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    if t.get_device() < 0:
        return contextlib.nullcontext()  # (refused by the call)
    handle = _stream(stream)
    # (1 is CUDA's other name of the default stream.)
    return torch.cuda.stream(torch.cuda.ExternalStream(0 if handle == 1 else handle, device=t.device))


def _call(torch, index, function, args, workspace=None, need=None) -> None:
    """function(*args, stream) with device `index` and its current stream; raises if it is
    refused. A function that takes a workspace before the stream has ``need``, the bytes it asks
    for: the caller's workspace or, for the length of the call, torch's allocator's on the very
    stream.

    The stream is read as its raw handle, and the allocator is called directly: a stream object
    costs 2.9 us of a call that takes 9, a tensor 7."""
    c = torch._C
    if index != c._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(torch, index, function, args, workspace, need)
    handle = c._cuda_getCurrentRawStream(index)
    if need is None:
        status = function(*args, handle)
    elif workspace is not None:
        if workspace.get_device() != index:
            raise ValueError(f"workspace is on {workspace.device}, not cuda:{index}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        status = function(*args, workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), handle)
    elif need == 0:
        status = function(*args, None, 0, handle)
    else:
        scratch = c._cuda_cudaCachingAllocator_raw_alloc(need, handle)
        try:
            status = function(*args, scratch, need, handle)
        finally:
            c._cuda_cudaCachingAllocator_raw_delete(scratch)
    if status:
        raise TpgemmError(status, tpgemm_last_error_detail())


def linear(A, W, bias=None, residual=None, *, act="none", scale_a=None, scale_w=None,
           out_dtype=None, out=None, pre=None, workspace=None, stream=None):
    """Y = act(scale_a[m] scale_w[n] A.W^T + bias) + residual on CUDA tensors; returns Y.

    A [M, K] and W [N, K] are both float16, bfloat16, float8_e4m3fn or float8_e5m2; Y, bias [N],
    residual [M, N] and ``pre`` [M, N] (given to receive the value before the activation) are of
    out_dtype (float16, bfloat16 or float32; by default A's 16-bit type, or bfloat16). The float32
    scales, per row of A and of W, are for the 8-bit types. act: none, relu, silu, gelu or
    gelu_tanh. Matrices may be row-strided; ``out`` may be the residual itself. The workspace, if
    one is needed (tpgemm_linear_workspace_bytes), is allocated here with torch unless given.
    stream (by default the current one) is current for the call: its memory holds the outputs."""
    if stream is not None:
        with _current(stream, A):
            return linear(A, W, bias, residual, act=act, scale_a=scale_a, scale_w=scale_w,
                          out_dtype=out_dtype, out=out, pre=pre, workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    M, K, index, device = _sizes("A", A)
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    N = W.shape[0]
    dt = A.dtype
    lda = _matrix("A", A, M, K, dt, index)
    ldw = _matrix("W", W, N, K, dt, index)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (dt if dt.itemsize == 2 else torch.bfloat16)
    act = _act_code(act)
    codes = elem_code(dt), elem_code(out_dtype), act
    if out is None:
        out, ldy = torch.empty((M, N), dtype=out_dtype, device=device), N
    else:
        ldy = _matrix("out", out, M, N, out_dtype, index)
    ldr = ldz = 0
    pr = pz = pb = psa = psw = None
    if residual is not None:
        ldr, pr = _matrix("residual", residual, M, N, out_dtype, index), residual.data_ptr()
    if pre is not None:
        ldz, pz = _matrix("pre", pre, M, N, out_dtype, index), pre.data_ptr()
    if bias is not None:
        pb = _vector("bias", bias, N, out_dtype, index)
    if scale_a is not None:
        psa = _vector("scale_a", scale_a, M, torch.float32, index)
    if scale_w is not None:
        psw = _vector("scale_w", scale_w, N, torch.float32, index)
    desc = ctypes.byref(LinearDesc(M, N, K, lda, ldw, ldr, ldy, ldz, *codes))
    pa, pw = A.data_ptr(), W.data_ptr()
    need = 0
    # (Operands whose rows start on 128-byte lines need no workspace: the library's promise.)
    if (pa | pw | (lda | ldw) * dt.itemsize) & 127:
        need = lib.tpgemm_linear_workspace_bytes(pa, pw, desc)
    _call(torch, index, lib.tpgemm_linear,
          (out.data_ptr(), pz, pa, pw, psa, psw, pb, pr, desc), workspace, need)
    return out


def linear_backward(dY, A, W, pre=None, *, act="none", grad_dtype=None, need=(True, True, True),
                    workspace=None, stream=None):
    """(dA, dW, dbias) of Y = act(A.W^T + bias) + residual, given dY [M, N] (the residual's own
    gradient) and ``pre``, the value before the activation (not needed for act="none").

    dY, A, W, pre and dA are all float16 or all bfloat16; dW and dbias are of grad_dtype (float32,
    float16 or bfloat16; by default A's type). ``need`` says which of the three are wanted; the
    others are None. stream: as for linear."""
    if stream is not None:
        with _current(stream, A):
            return linear_backward(dY, A, W, pre, act=act, grad_dtype=grad_dtype, need=need,
                                   workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    M, K, index, device = _sizes("A", A)
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    N = W.shape[0]
    dt = A.dtype
    grad_dtype = dt if grad_dtype is None else grad_dtype
    code = _act_code(act)
    ldz, pz = 0, None
    if code != TPGEMM_ACT_NONE:
        if pre is None:
            raise ValueError(f"act={act!r} needs pre, the value before the activation")
        ldz, pz = _matrix("pre", pre, M, N, dt, index), pre.data_ptr()
    desc = ctypes.byref(LinearGradDesc(
        M, N, K, _matrix("dY", dY, M, N, dt, index), ldz, _matrix("A", A, M, K, dt, index),
        _matrix("W", W, N, K, dt, index), K, K, elem_code(dt), elem_code(grad_dtype), code))
    dA = dW = dbias = pda = pdw = pdb = None
    if need[0]:
        dA = torch.empty((M, K), dtype=dt, device=device)
        pda = dA.data_ptr()
    if need[1]:
        dW = torch.empty((N, K), dtype=grad_dtype, device=device)
        pdw = dW.data_ptr()
    if need[2]:
        dbias = torch.empty(N, dtype=grad_dtype, device=device)
        pdb = dbias.data_ptr()
    py, pa, pw = dY.data_ptr(), A.data_ptr(), W.data_ptr()
    _call(torch, index, lib.tpgemm_linear_backward, (pda, pdw, pdb, py, pa, pw, pz, desc),
          workspace, lib.tpgemm_linear_backward_workspace_bytes(py, pa, pw, desc))
    return dA, dW, dbias


def _gated_sizes(A, W):
    M, K, index, device = _sizes("A", A)
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    if W.shape[0] % 2:
        raise ValueError(f"W must hold two projections of as many rows, got {W.shape[0]}")
    return M, K, W.shape[0] // 2, index, device


def gated_linear(A, W, bias=None, *, act="silu", scale_a=None, scale_w=None, out_dtype=None, out=None,
                 pre=None, workspace=None, stream=None):
    """Y = act(G) U, [G | U] = scale_a[m] scale_w[n] A.W^T + bias on CUDA tensors; returns Y.

    A is [M, K] and W [2N, K]: the gate's N rows, then those of the factor U. Y is [M, N], bias and
    scale_w [2N], and ``pre`` [M, 2N] is given to receive [G | U], which gated_linear_backward
    needs. Types, scales, activations, strides, workspace (tpgemm_gated_linear_workspace_bytes) and
    stream are as for linear."""
    if stream is not None:
        with _current(stream, A):
            return gated_linear(A, W, bias, act=act, scale_a=scale_a, scale_w=scale_w,
                                out_dtype=out_dtype, out=out, pre=pre, workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    M, K, N, index, device = _gated_sizes(A, W)
    dt = A.dtype
    lda = _matrix("A", A, M, K, dt, index)
    ldw = _matrix("W", W, 2 * N, K, dt, index)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (dt if dt.itemsize == 2 else torch.bfloat16)
    codes = elem_code(dt), elem_code(out_dtype), _act_code(act)
    if out is None:
        out, ldy = torch.empty((M, N), dtype=out_dtype, device=device), N
    else:
        ldy = _matrix("out", out, M, N, out_dtype, index)
    ldz = 0
    pz = pb = psa = psw = None
    if pre is not None:
        ldz, pz = _matrix("pre", pre, M, 2 * N, out_dtype, index), pre.data_ptr()
    if bias is not None:
        pb = _vector("bias", bias, 2 * N, out_dtype, index)
    if scale_a is not None:
        psa = _vector("scale_a", scale_a, M, torch.float32, index)
    if scale_w is not None:
        psw = _vector("scale_w", scale_w, 2 * N, torch.float32, index)
    desc = ctypes.byref(LinearDesc(M, N, K, lda, ldw, 0, ldy, ldz, *codes))
    pa, pw = A.data_ptr(), W.data_ptr()
    need = 0
    # (Operands whose rows start on 128-byte lines need no workspace: the library's promise.)
    if (pa | pw | (lda | ldw) * dt.itemsize) & 127:
        need = lib.tpgemm_gated_linear_workspace_bytes(pa, pw, desc)
    _call(torch, index, lib.tpgemm_gated_linear,
          (out.data_ptr(), pz, pa, pw, psa, psw, pb, desc), workspace, need)
    return out


def gated_linear_backward(dY, A, W, pre, *, act="silu", grad_dtype=None, need=(True, True, True),
                          workspace=None, stream=None):
    """(dA, dW, dbias) of Y = act(G) U, [G | U] = A.W^T + bias, given dY [M, N] and ``pre`` [M, 2N],
    which holds [G | U]. W and dW are [2N, K], dbias [2N]; the rest is as for linear_backward."""
    if stream is not None:
        with _current(stream, A):
            return gated_linear_backward(dY, A, W, pre, act=act, grad_dtype=grad_dtype, need=need,
                                         workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    M, K, N, index, device = _gated_sizes(A, W)
    dt = A.dtype
    grad_dtype = dt if grad_dtype is None else grad_dtype
    desc = ctypes.byref(LinearGradDesc(
        M, N, K, _matrix("dY", dY, M, N, dt, index), _matrix("pre", pre, M, 2 * N, dt, index),
        _matrix("A", A, M, K, dt, index), _matrix("W", W, 2 * N, K, dt, index), K, K,
        elem_code(dt), elem_code(grad_dtype), _act_code(act)))
    dA = dW = dbias = pda = pdw = pdb = None
    if need[0]:
        dA = torch.empty((M, K), dtype=dt, device=device)
        pda = dA.data_ptr()
    if need[1]:
        dW = torch.empty((2 * N, K), dtype=grad_dtype, device=device)
        pdw = dW.data_ptr()
    if need[2]:
        dbias = torch.empty(2 * N, dtype=grad_dtype, device=device)
        pdb = dbias.data_ptr()
    py, pa, pw = dY.data_ptr(), A.data_ptr(), W.data_ptr()
    _call(torch, index, lib.tpgemm_gated_linear_backward,
          (pda, pdw, pdb, py, pa, pw, pre.data_ptr(), desc), workspace,
          lib.tpgemm_gated_linear_backward_workspace_bytes(py, pa, pw, desc))
    return dA, dW, dbias


class RmsNorm(typing.NamedTuple):
    """What rmsnorm returns; what was not asked for is None."""
    y: object
    h: object      # x + residual
    scale: object  # float32 [rows] ("row") or uint8 [rows, ceil(cols / 32)] E8M0 ("mx")
    rstd: object   # float32 [rows]


def rmsnorm(x, weight, residual=None, *, eps=1e-6, quant=None, out_dtype=None, need_rstd=False,
            out=None, out_h=None, stream=None):
    """Root-mean-square norm of the rows of h = x + residual: y = h / sqrt(mean(h^2) + eps) weight.

    x, residual and h [rows, cols] are float16, bfloat16 or float32; weight [cols] is of x's type
    or float32. y is of out_dtype: a float type (by default x's), or with quant="row" (one float32
    scale per row, linear's scale_a) or quant="mx" (one E8M0 scale per 32 columns, gemm_mx's SFA)
    float8_e4m3fn (the default) or float8_e5m2, holding y / scale. h is returned with a residual
    only; it may be written in place (out_h = x or residual). stream: as for linear."""
    if stream is not None:
        with _current(stream, x):
            return rmsnorm(x, weight, residual, eps=eps, quant=quant, out_dtype=out_dtype,
                           need_rstd=need_rstd, out=out, out_h=out_h)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    rows, cols, index, device = _sizes("x", x)
    dt = x.dtype
    if quant not in _SCALES:
        raise ValueError(f"quant must be None, 'row' or 'mx', got {quant!r}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (dt if quant is None else torch.float8_e4m3fn)
    wt = weight.dtype
    if wt is not dt and wt is not torch.float32:
        raise TypeError(f"weight must be {dt} or float32, got {wt}")
    pg = _vector("weight", weight, cols, wt, index)
    ldx = _matrix("x", x, rows, cols, dt, index)
    codes = elem_code(dt), elem_code(wt), elem_code(out_dtype), _SCALES[quant]
    if out is None:
        out, ldy = torch.empty((rows, cols), dtype=out_dtype, device=device), cols
    else:
        ldy = _matrix("out", out, rows, cols, out_dtype, index)
    h = scale = rstd = pr = ph = ps = prstd = None
    ldr = ldh = 0
    if residual is not None:
        ldr, pr = _matrix("residual", residual, rows, cols, dt, index), residual.data_ptr()
        if out_h is None:
            h, ldh = torch.empty((rows, cols), dtype=dt, device=device), cols
        else:
            h, ldh = out_h, _matrix("out_h", out_h, rows, cols, dt, index)
        ph = h.data_ptr()
    elif out_h is not None:
        raise ValueError("out_h needs a residual (h is x without one)")
    if quant == "row":
        scale = torch.empty(rows, dtype=torch.float32, device=device)
        ps = scale.data_ptr()
    elif quant == "mx":
        scale = torch.empty((rows, (cols + 31) // 32), dtype=torch.uint8, device=device)
        ps = scale.data_ptr()
    if need_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
        prstd = rstd.data_ptr()
    desc = RmsNormDesc(rows, cols, ldx, ldr, ldh, ldy, *codes, eps)
    _call(torch, index, lib.tpgemm_rmsnorm,
          (out.data_ptr(), ph, ps, prstd, x.data_ptr(), pr, pg, ctypes.byref(desc)))
    return RmsNorm(out, h, scale, rstd)


def rmsnorm_backward(dy, h, rstd, weight, dh=None, *, grad_dtype=None, need=(True, True), out=None,
                     workspace=None, stream=None):
    """(dx, dweight) of a root-mean-square norm, given dy, the normalised rows' h and rstd, and the
    gradient dh that reaches h past the norm (or None). dx is the gradient of x and of residual.

    dy, h, dh and dx [rows, cols] are of one type (float16, bfloat16 or float32), dweight of
    grad_dtype (by default weight's). ``need`` says which are wanted; ``out`` may be dy, h or dh.
    stream: as for linear."""
    if stream is not None:
        with _current(stream, dy):
            return rmsnorm_backward(dy, h, rstd, weight, dh, grad_dtype=grad_dtype, need=need,
                                    out=out, workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    rows, cols, index, device = _sizes("dy", dy)
    dt, wt = dy.dtype, weight.dtype
    grad_dtype = wt if grad_dtype is None else grad_dtype
    if wt is not dt and wt is not torch.float32:
        raise TypeError(f"weight must be {dt} or float32, got {wt}")
    pg = _vector("weight", weight, cols, wt, index)
    prstd = _vector("rstd", rstd, rows, torch.float32, index)
    dx = dweight = pdx = pdw = pdh = None
    lddh = lddx = scratch = 0
    if dh is not None:
        lddh, pdh = _matrix("dh", dh, rows, cols, dt, index), dh.data_ptr()
    if need[0]:
        if out is None:
            dx, lddx = torch.empty((rows, cols), dtype=dt, device=device), cols
        else:
            dx, lddx = out, _matrix("out", out, rows, cols, dt, index)
        pdx = dx.data_ptr()
    desc = RmsNormGradDesc(rows, cols, _matrix("dy", dy, rows, cols, dt, index),
                           _matrix("h", h, rows, cols, dt, index), lddh, lddx, elem_code(dt),
                           elem_code(wt), elem_code(grad_dtype))
    if need[1]:
        dweight = torch.empty(cols, dtype=grad_dtype, device=device)
        pdw = dweight.data_ptr()
        scratch = lib.tpgemm_rmsnorm_backward_workspace_bytes(rows, cols)
    _call(torch, index, lib.tpgemm_rmsnorm_backward,
          (pdx, pdw, dy.data_ptr(), h.data_ptr(), prstd, pg, pdh, ctypes.byref(desc)), workspace,
          scratch)
    return dx, dweight


class Dropout(typing.NamedTuple):
    """A dropout's numbers. The mask is a function of these and of each element's row and column
    (Philox4x32-10, see include/tpgemm.h), so the backward pass is given the same ones."""
    p: float          # probability to drop an element, in [0, 1)
    seed: int         # below 2^64
    offset: object = 0  # below 2^64, or a CUDA int64 tensor of one element, read when the work runs


def _drop(d, index):
    """The members of the tpgemm_drop of a Dropout (or of None: nothing is dropped)."""
    if d is None:
        return ()
    p, seed, offset = d
    counter = None
    if not isinstance(offset, int):
        torch = _torch or _import_torch()
        if not isinstance(offset, torch.Tensor):
            raise TypeError(f"offset must be an int or a tensor, got {type(offset).__name__}")
        if offset.dtype is not torch.int64 or offset.numel() != 1 or offset.get_device() != index:
            raise ValueError(f"offset must be an int64 tensor of one element on cuda:{index}")
        offset, counter = 0, offset.data_ptr()
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset must be at least 0 and below 2^64")
    return p, seed, offset, counter


def dropout(x, drop, residual=None, *, out=None, stream=None):
    """y = x / (1 - p) where it is kept and 0 where it is dropped, plus residual; returns y.

    x, residual and y [rows, cols] are float16, bfloat16 or float32; drop is a Dropout. ``out`` may
    be x or residual itself. stream: as for linear."""
    if stream is not None:
        with _current(stream, x):
            return dropout(x, drop, residual, out=out)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    rows, cols, index, device = _sizes("x", x)
    dt = x.dtype
    ldx = _matrix("x", x, rows, cols, dt, index)
    code = elem_code(dt)
    pr, ldr = None, 0
    if residual is not None:
        ldr, pr = _matrix("residual", residual, rows, cols, dt, index), residual.data_ptr()
    if out is None:
        # (Like a dense x: that is a third of a microsecond faster.)
        out, ldy = torch.empty_like(x) if ldx == cols else torch.empty((rows, cols), dtype=dt, device=device), cols
    else:
        ldy = _matrix("out", out, rows, cols, dt, index)
    desc = DropoutDesc(rows, cols, ldx, ldr, ldy, code, *_drop(drop, index))
    _call(torch, index, lib.tpgemm_dropout,
          (out.data_ptr(), x.data_ptr(), pr, ctypes.byref(desc)))
    return out


def dropout_backward(dy, drop, *, out=None, stream=None):
    """The gradient of dropout's x, given that of y and the same Dropout (the residual's is dy).
    ``out`` may be dy itself. stream: as for linear."""
    return dropout(dy, drop, out=out, stream=stream)


class LayerNorm(typing.NamedTuple):
    """What layernorm returns; what was not asked for is None."""
    y: object
    h: object      # dropout(x) + residual
    scale: object  # float32 [rows] ("row")
    mean: object   # float32 [rows]
    rstd: object   # float32 [rows]


def layernorm(x, weight, bias=None, residual=None, *, eps=1e-5, dropout=None, quant=None,
              out_dtype=None, need_stats=False, out=None, out_h=None, stream=None):
    """Layer norm of the rows of h = dropout(x) + residual:
    y = (h - mean(h)) / sqrt(var(h) + eps) weight + bias.

    x, residual and h [rows, cols] are float16, bfloat16 or float32; weight and bias [cols] are of
    x's type or both float32; dropout is a Dropout or None. y is of out_dtype: a float type (by
    default x's), or with quant="row" (one float32 scale per row, linear's scale_a) float8_e4m3fn
    (the default) or float8_e5m2, holding y / scale. h is returned with a residual or a dropout
    only; it may be written in place (out_h = x or residual). need_stats: mean and rstd are
    returned, for layernorm_backward. stream: as for linear."""
    if stream is not None:
        with _current(stream, x):
            return layernorm(x, weight, bias, residual, eps=eps, dropout=dropout, quant=quant,
                             out_dtype=out_dtype, need_stats=need_stats, out=out, out_h=out_h)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    rows, cols, index, device = _sizes("x", x)
    dt = x.dtype
    if quant not in (None, "row"):
        raise ValueError(f"quant must be None or 'row', got {quant!r}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (dt if quant is None else torch.float8_e4m3fn)
    wt = weight.dtype
    if wt is not dt and wt is not torch.float32:
        raise TypeError(f"weight must be {dt} or float32, got {wt}")
    pg = _vector("weight", weight, cols, wt, index)
    pb = None if bias is None else _vector("bias", bias, cols, wt, index)
    ldx = _matrix("x", x, rows, cols, dt, index)
    codes = elem_code(dt), elem_code(wt), elem_code(out_dtype), _SCALES[quant]
    if out is None:
        if out_dtype is dt and ldx == cols:  # (faster)
            out, ldy = torch.empty_like(x), cols
        else:
            out, ldy = torch.empty((rows, cols), dtype=out_dtype, device=device), cols
    else:
        ldy = _matrix("out", out, rows, cols, out_dtype, index)
    h = scale = mean = rstd = pr = ph = ps = pm = prstd = None
    ldr = ldh = 0
    if residual is not None:
        ldr, pr = _matrix("residual", residual, rows, cols, dt, index), residual.data_ptr()
    if residual is not None or dropout is not None:
        if out_h is None:
            h, ldh = torch.empty_like(x) if ldx == cols else torch.empty((rows, cols), dtype=dt, device=device), cols
        else:
            h, ldh = out_h, _matrix("out_h", out_h, rows, cols, dt, index)
        ph = h.data_ptr()
    elif out_h is not None:
        raise ValueError("out_h needs a residual or a dropout (h is x without them)")
    if quant == "row":
        scale = torch.empty(rows, dtype=torch.float32, device=device)
        ps = scale.data_ptr()
    if need_stats:
        mean = torch.empty(rows, dtype=torch.float32, device=device)
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
        pm, prstd = mean.data_ptr(), rstd.data_ptr()
    desc = LayerNormDesc(rows, cols, ldx, ldr, ldh, ldy, *codes, eps, *_drop(dropout, index))
    _call(torch, index, lib.tpgemm_layernorm,
          (out.data_ptr(), ph, ps, pm, prstd, x.data_ptr(), pr, pg, pb, ctypes.byref(desc)))
    return LayerNorm(out, h, scale, mean, rstd)


class LayerNormGrad(typing.NamedTuple):
    """What layernorm_backward returns; what was not asked for is None."""
    dx: object
    dresidual: object  # dx itself without a dropout
    dweight: object
    dbias: object


def layernorm_backward(dy, h, mean, rstd, weight, dh=None, *, dropout=None, grad_dtype=None,
                       need=(True, True, True, True), out=None, workspace=None, stream=None):
    """The gradients of a layer norm, given dy, the normalised rows' h, mean and rstd, the gradient
    dh that reaches h past the norm (or None), and the Dropout of the forward pass.

    dy, h, dh, dx and dresidual [rows, cols] are of one type (float16, bfloat16 or float32),
    dweight and dbias of grad_dtype (by default weight's). ``need`` says which of dx, dresidual,
    dweight and dbias are wanted; ``out`` (of dx, or of both without a dropout) may be dy, h or dh, and
    is refused where it would not be written. stream: as for linear."""
    apart = dropout is not None
    dx_wanted = need[0] or (need[1] and not apart)
    if out is not None and not dx_wanted:
        raise ValueError("out is dx's, which need leaves out")
    if stream is not None:
        with _current(stream, dy):
            return layernorm_backward(dy, h, mean, rstd, weight, dh, dropout=dropout,
                                      grad_dtype=grad_dtype, need=need, out=out,
                                      workspace=workspace)
    torch = _torch or _import_torch()
    lib = _lib or _load()
    rows, cols, index, device = _sizes("dy", dy)
    dt, wt = dy.dtype, weight.dtype
    grad_dtype = wt if grad_dtype is None else grad_dtype
    if wt is not dt and wt is not torch.float32:
        raise TypeError(f"weight must be {dt} or float32, got {wt}")
    pg = _vector("weight", weight, cols, wt, index)
    pm = _vector("mean", mean, rows, torch.float32, index)
    prstd = _vector("rstd", rstd, rows, torch.float32, index)
    dx = dr = pdh = pdx = pdr = pdw = pdb = dweight = dbias = None
    lddh = lddx = lddr = scratch = 0
    if dh is not None:
        lddh, pdh = _matrix("dh", dh, rows, cols, dt, index), dh.data_ptr()
    lddy = _matrix("dy", dy, rows, cols, dt, index)
    if dx_wanted:
        if out is None:
            dx, lddx = torch.empty_like(dy) if lddy == cols else torch.empty((rows, cols), dtype=dt, device=device), cols
        else:
            dx, lddx = out, _matrix("out", out, rows, cols, dt, index)
        pdx = dx.data_ptr()
    if need[1] and apart:
        dr, lddr = torch.empty_like(dy) if lddy == cols else torch.empty((rows, cols), dtype=dt, device=device), cols
        pdr = dr.data_ptr()
    if need[2]:
        dweight = torch.empty(cols, dtype=grad_dtype, device=device)
        pdw = dweight.data_ptr()
    if need[3]:
        dbias = torch.empty(cols, dtype=grad_dtype, device=device)
        pdb = dbias.data_ptr()
    if need[2] or need[3]:
        scratch = lib.tpgemm_layernorm_backward_workspace_bytes(rows, cols)
    desc = LayerNormGradDesc(rows, cols, lddy,
                             _matrix("h", h, rows, cols, dt, index), lddh, lddx, lddr, elem_code(dt),
                             elem_code(wt), elem_code(grad_dtype), *_drop(dropout, index))
    _call(torch, index, lib.tpgemm_layernorm_backward,
          (pdx, pdr, pdw, pdb, dy.data_ptr(), h.data_ptr(), pm, prstd, pg, pdh, ctypes.byref(desc)),
          workspace, scratch)
    if not apart:
        dr = dx if need[1] else None
        dx = dx if need[0] else None
    return LayerNormGrad(dx, dr, dweight, dbias)
