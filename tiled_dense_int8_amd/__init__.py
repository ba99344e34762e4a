"""Python binding of libtdi8.so, the gfx950 tiled int8 GEMM library.

Argument marshalling only: every step of the product runs in the library's
HIP kernels (C ABI in include/tdi8.h).  The names mirror the C entry points;
``gemm`` is a convenience wrapper that takes torch tensors, whose only role
is device memory and the current stream.

There is no fallback: if libtdi8.so is missing or fails to load, importing this
package raises.  Build it with ``python tiled_dense_int8_amd/build.py`` (or
``__graft_entry__.build()``).  The module _calls only shortens the calls of the
8-bit layer operators: where it is missing, or was built against another torch,
importing warns, and they call the same kernels by way of Python.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch  # loads torch's HIP runtime first, so the library binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtdi8.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with tiled_dense_int8_amd/build.py")
_lib = ctypes.CDLL(LIB_PATH)
try:
    from . import _calls
    if _calls.torch_version != str(torch.__version__):
        raise ImportError(f"it was built against torch {_calls.torch_version}, this is {torch.__version__}")
except ImportError as e:
    _calls = None
    warnings.warn(f"{_HERE}/_calls.so cannot be used ({e}): calls of the 8-bit layer operators take longer; "
                  "build it with tiled_dense_int8_amd/build.py", RuntimeWarning)

OK = 0
ERR_INVALID_VALUE = -1
ERR_NULL_POINTER = -2
ERR_ALIASING = -3
ERR_UNSUPPORTED_DEVICE = -4
ERR_BAD_CONFIG = -5
ERR_HIP = -6

F32, BF16, F16 = 0, 1, 2  # tdi8_type

ROUTE_GENERAL, ROUTE_FALLBACK, ROUTE_SKINNY = 0, 1, 2


class TileConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "id", "family", "mfma_m", "mfma_n", "mfma_k", "waves_m", "waves_n", "waves_k",
        "m_tiles", "n_tiles", "block_m", "block_n", "block_k", "stages", "threads", "lds_bytes",
        "vgprs", "agprs", "blocks_per_cu", "reuse1_id", "excluded", "sgprs")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


class HwInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_cu", "max_threads_per_block", "min_active_threads", "skinny_max_m")]


class Selection(ctypes.Structure):
    _fields_ = [("id", ctypes.c_int), ("route", ctypes.c_int), ("survivors", ctypes.c_int * 5)]


FORM_NONE, FORM_PREDICATED, FORM_PIPELINED, FORM_PIPELINED_EDGE, FORM_SPLIT, FORM_SPLIT_EDGE, \
    FORM_SKINNY_DMA, FORM_SKINNY_PREDICATED, FORM_SKINNY_ROW_GROUPS, FORM_PREDICATED_PREFETCH, \
    FORM_PERSISTENT = range(11)


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "config_id", "form", "splits", "kernels", "grid_x", "grid_y", "threads")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


SCALED_NONE, SCALED_STREAM, SCALED_STREAM_UNALIGNED, SCALED_LDS, SCALED_STAGED = range(5)


class ScaledPlan(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int), ("block_m", ctypes.c_int), ("block_n", ctypes.c_int),
                ("threads", ctypes.c_int), ("blocks", ctypes.c_int64)]


_i, _p, _f = ctypes.c_int, ctypes.c_void_p, ctypes.c_float
_GEMM_ARGS = [_i, _i, _i, _p, _i, _p, _i, _p, _i, _p]
_SIGNATURES = {
    "gemm_s8s8s32": (_i, _GEMM_ARGS),
    "gemm_s8s8s32_bt": (_i, _GEMM_ARGS),
    "gemm_s8s8s32_with_config": (_i, [_i, _i] + _GEMM_ARGS),
    "gemm_s8s8s32_persistent": (_i, [_i, _i] + _GEMM_ARGS[:-1] + [_i, _GEMM_ARGS[-1]]),
    "select_tile_config": (_i, [_i, _i, _i]),
    "tile_config_count": (_i, []),
    "tile_config_info": (_i, [_i, ctypes.POINTER(TileConfig)]),
    "tile_config_split_k": (_i, [_i, _i, _i, _i, _i]),
    "gemm_plan": (_i, [_i, _i, _i, _i, _i, _p, _i, _p, _i, _p, _i, ctypes.POINTER(Plan)]),
    "select_tile_config_for": (_i, [_i, _i, _i, ctypes.POINTER(HwInfo), ctypes.POINTER(_i),
                                    ctypes.POINTER(Selection)]),
    "tdi8_validate": (_i, [_i, _i, _i, _i, _p, _i, _p, _i, _p, _i]),
    "conv2d_s8s8s32_nhwc": (_i, [_i] * 13 + [_p, _p, _p, _p]),
    "conv2d_s8s8s32_nhwc_with_config": (_i, [_i] * 14 + [_p, _p, _p, _p]),
    "conv2d_select_config": (_i, [_i] * 13),
    "conv2d_output_extent": (_i, [_i] * 5),
    "conv2d_validate": (_i, [_i] * 13 + [_p, _p, _p]),
    "rmsnorm_quant_s8": (_i, [_i] * 3 + [_p, _i, _p, _i, _p, _f, _p, _i, _p, _i, _p, _p]),
    "rmsnorm_quant_f8": (_i, [_i] * 3 + [_p, _i, _p, _i, _p, _f, _p, _i, _p, _i, _p, _i, _p]),
    "swiglu_quant_s8": (_i, [_i] * 3 + [_p, _i, _p, _i, _p, _i, _p, _p]),
    "swiglu_quant_f8": (_i, [_i] * 3 + [_p, _i, _p, _i, _p, _i, _p, _i, _p]),
    "gemm_s8s8_grouped": (_i, [_i] * 5 + [_p, _i, _i, _p, _p, _p, _p, _i, ctypes.c_int64, _p, _p, _i, _p]),
    "gemm_f8f8_block128": (_i, [_i] * 4 + [_p, _i, _p, _i, _p, _i, _p, _i, _p, _i, _p]),
    "scaled_product_plan": (_i, [_i] * 8 + [ctypes.POINTER(ScaledPlan)]),
    "tdi8_status_string": (ctypes.c_char_p, [_i]),
    "tdi8_last_hip_error": (_i, []),
    "tdi8_kernel_code_hash": (ctypes.c_char_p, []),
    "tdi8_layer_code_hash": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGNATURES)


def load_library(path: str) -> ctypes.CDLL:
    """Another build of the same C ABI (the instrumented libtdi8_stamps.so),
    loaded beside libtdi8.so with the same signatures; its functions take the
    arguments of the module-level ones of the same name."""
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


class TDI8Error(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        msg = tdi8_status_string(status)
        if status == ERR_HIP:
            msg += f" (hipError_t {tdi8_last_hip_error()})"
        super().__init__(f"tdi8 status {status}: {msg}")


INT_MAX = 2 ** 31 - 1


def _int32(**vals) -> None:
    """The C entry points take int arguments; ctypes would wrap a larger
    Python int silently (2**32 + 5 arrives as 5), so refuse it here."""
    for name, v in vals.items():
        if not -2 ** 31 <= int(v) <= INT_MAX:
            raise ValueError(f"{name} = {v} does not fit the library's int arguments (|value| < 2**31)")


# ----- the C entry points, same names and arguments -------------------------------

def gemm_s8s8s32(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    _int32(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return _lib.gemm_s8s8s32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_s8s8s32_bt(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    _int32(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return _lib.gemm_s8s8s32_bt(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_s8s8s32_with_config(config_id, b_col_major, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    _int32(config_id=config_id, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return _lib.gemm_s8s8s32_with_config(config_id, 1 if b_col_major else 0, M, N, K, A, lda, B, ldb,
                                         C, ldc, stream)


def gemm_s8s8s32_persistent(config_id, b_col_major, M, N, K, A, lda, B, ldb, C, ldc, blocks=0, stream=0) -> int:
    _int32(config_id=config_id, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc, blocks=blocks)
    return _lib.gemm_s8s8s32_persistent(config_id, 1 if b_col_major else 0, M, N, K, A, lda, B, ldb,
                                        C, ldc, blocks, stream)


def gemm_plan(config_id, b_col_major, M, N, K, A, lda, B, ldb, C, ldc) -> Plan:
    """What the gemm call with these arguments would enqueue (config_id -1:
    the selected configuration); raises TDI8Error on a bad argument."""
    _int32(config_id=config_id, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    out = Plan()
    st = _lib.gemm_plan(config_id, 1 if b_col_major else 0, M, N, K, A, lda, B, ldb, C, ldc,
                        ctypes.byref(out))
    if st != OK:
        raise TDI8Error(st)
    return out


def select_tile_config(M, N, K) -> int:
    _int32(M=M, N=N, K=K)
    return _lib.select_tile_config(M, N, K)


def tile_config_split_k(config_id, M, N, K, num_cu) -> int:
    _int32(config_id=config_id, M=M, N=N, K=K, num_cu=num_cu)
    return _lib.tile_config_split_k(config_id, M, N, K, num_cu)


def tile_config_count() -> int:
    return _lib.tile_config_count()


def tile_config_info(config_id: int) -> TileConfig:
    out = TileConfig()
    st = _lib.tile_config_info(config_id, ctypes.byref(out))
    if st != OK:
        raise TDI8Error(st)
    return out


def select_tile_config_for(M, N, K, hw: HwInfo, blocks_per_cu) -> Selection:
    _int32(M=M, N=N, K=K)
    arr = (ctypes.c_int * tile_config_count())(*blocks_per_cu)
    out = Selection()
    st = _lib.select_tile_config_for(M, N, K, ctypes.byref(hw), arr, ctypes.byref(out))
    if st < 0:
        raise TDI8Error(st)
    return out


def tdi8_validate(b_col_major, M, N, K, A, lda, B, ldb, C, ldc) -> int:
    _int32(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    return _lib.tdi8_validate(1 if b_col_major else 0, M, N, K, A, lda, B, ldb, C, ldc)


def tdi8_status_string(status: int) -> str:
    return _lib.tdi8_status_string(status).decode()


def tdi8_last_hip_error() -> int:
    return _lib.tdi8_last_hip_error()


def tdi8_kernel_code_hash() -> str:
    return _lib.tdi8_kernel_code_hash().decode()


def tdi8_layer_code_hash() -> str:
    return _lib.tdi8_layer_code_hash().decode()


# ----- torch convenience -----------------------------------------------------------

def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _device_of(*tensors) -> "torch.device":
    """The one GPU holding every tensor (the kernels dereference their data
    pointers as device addresses, so host tensors must never reach them)."""
    devs = {t.device for t in tensors}
    if any(d.type != "cuda" for d in devs):
        raise ValueError("tensors must be on a GPU")
    if len(devs) != 1:
        raise ValueError(f"tensors are on different devices: {sorted(str(d) for d in devs)}")
    return devs.pop()


def gemm(A: "torch.Tensor", B: "torch.Tensor", b_col_major: bool, out: "torch.Tensor | None" = None,
         config: int | None = None, stream=None, persistent_blocks: int | None = None) -> "torch.Tensor":
    """C = A x B on the GPU.

    A: int8 (M, K) with unit column stride (row stride = lda).
    B: int8 storage of the logical K x N matrix: (K, N) row-major if
       b_col_major is False, (N, K) with K contiguous if True.
    out: optional int32 (M, N) with unit column stride (row stride = ldc).
    config: run this configuration id instead of the selected one.
    persistent_blocks: run the persistent whole-tile form with this many
       blocks (0: one wave of resident blocks); needs whole tiles.
    """
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    if A.dim() != 2 or B.dim() != 2 or A.stride(1) != 1 or B.stride(1) != 1:
        raise ValueError("A and B must be 2-D with unit column stride")
    M, K = A.shape
    N = B.shape[0] if b_col_major else B.shape[1]
    if (B.shape[1] if b_col_major else B.shape[0]) != K:
        raise ValueError("inner dimensions differ")
    dev = _device_of(A, B) if out is None else _device_of(A, B, out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32, device=dev)
    if out.dtype != torch.int32 or out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError("out must be int32 (M, N) with unit column stride")
    lda, ldb, ldc = max(A.stride(0), 1), max(B.stride(0), 1), max(out.stride(0), 1)
    _int32(M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc)
    with torch.cuda.device(dev):
        s = _stream_handle(stream)
        if persistent_blocks is not None:
            st = gemm_s8s8s32_persistent(-1 if config is None else config, b_col_major, M, N, K, A.data_ptr(),
                                         lda, B.data_ptr(), ldb, out.data_ptr(), ldc, persistent_blocks, s)
        elif config is None:
            fn = gemm_s8s8s32_bt if b_col_major else gemm_s8s8s32
            st = fn(M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc, s)
        else:
            st = gemm_s8s8s32_with_config(config, b_col_major, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                                          out.data_ptr(), ldc, s)
    if st != OK:
        raise TDI8Error(st)
    return out


# ---- convolution ---------------------------------------------------------------

def _conv_int32(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w) -> None:
    _int32(N=N, H=H, W=W, C=C, K=K, R=R, S=S, pad_h=pad_h, pad_w=pad_w, stride_h=stride_h,
           stride_w=stride_w, dil_h=dil_h, dil_w=dil_w)


def conv2d_s8s8s32_nhwc(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w,
                        x, w, y, stream=0) -> int:
    _conv_int32(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w)
    return _lib.conv2d_s8s8s32_nhwc(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w,
                                    x, w, y, stream)


def conv2d_s8s8s32_nhwc_with_config(config_id, N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w,
                                    dil_h, dil_w, x, w, y, stream=0) -> int:
    _int32(config_id=config_id)
    _conv_int32(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w)
    return _lib.conv2d_s8s8s32_nhwc_with_config(config_id, N, H, W, C, K, R, S, pad_h, pad_w, stride_h,
                                                stride_w, dil_h, dil_w, x, w, y, stream)


def conv2d_select_config(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w) -> int:
    _conv_int32(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w)
    return _lib.conv2d_select_config(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w)


def conv2d_output_extent(H, R, pad, stride, dil) -> int:
    _int32(H=H, R=R, pad=pad, stride=stride, dil=dil)
    return _lib.conv2d_output_extent(H, R, pad, stride, dil)


def conv2d_validate(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w, x, w, y) -> int:
    _conv_int32(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w)
    return _lib.conv2d_validate(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w, x, w, y)


def conv2d(x, w, pad=(0, 0), stride=(1, 1), dil=(1, 1), out=None, config=None, stream=None):
    """y = conv2d(x, w) for torch tensors on the GPU: x int8 N x H x W x C,
    w int8 K x R x S x C (both contiguous), y int32 N x P x Q x K."""
    if x.dtype != torch.int8 or w.dtype != torch.int8:
        raise TypeError("x and w must be int8")
    if x.dim() != 4 or w.dim() != 4 or not x.is_contiguous() or not w.is_contiguous():
        raise ValueError("x (N, H, W, C) and w (K, R, S, C) must be contiguous 4-D tensors")
    N, H, W, C = x.shape
    K, R, S, Cw = w.shape
    if Cw != C:
        raise ValueError(f"channel counts differ: x has {C}, w has {Cw}")
    P = conv2d_output_extent(H, R, pad[0], stride[0], dil[0])
    Q = conv2d_output_extent(W, S, pad[1], stride[1], dil[1])
    if P < 0 or Q < 0:
        raise TDI8Error(min(P, Q))
    dev = _device_of(x, w) if out is None else _device_of(x, w, out)
    if out is None:
        out = torch.empty((N, P, Q, K), dtype=torch.int32, device=dev)
    if out.dtype != torch.int32 or tuple(out.shape) != (N, P, Q, K) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous int32 tensor of shape {(N, P, Q, K)}")
    with torch.cuda.device(dev):
        args = (N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1], dil[0], dil[1],
                x.data_ptr(), w.data_ptr(), out.data_ptr(), _stream_handle(stream))
        st = conv2d_s8s8s32_nhwc(*args) if config is None else conv2d_s8s8s32_nhwc_with_config(config, *args)
    if st != OK:
        raise TDI8Error(st)
    return out


# ---- 8-bit operands of a layer: norm and gated activation ---------------------------

_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
BLOCK = 128  # columns that share a scale in the f8 format


def rmsnorm_quant_s8(type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, stream=0) -> int:
    _int32(type=type, T=T, H=H, ldx=ldx, ldr=ldr, ldsum=ldsum, ldq=ldq)
    return _lib.rmsnorm_quant_s8(type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, stream)


def rmsnorm_quant_f8(type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, lds,
                     stream=0) -> int:
    _int32(type=type, T=T, H=H, ldx=ldx, ldr=ldr, ldsum=ldsum, ldq=ldq, lds=lds)
    return _lib.rmsnorm_quant_f8(type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, lds,
                                 stream)


def swiglu_quant_s8(type, T, N, gate, ldg, up, ldu, q, ldq, scale, stream=0) -> int:
    _int32(type=type, T=T, N=N, ldg=ldg, ldu=ldu, ldq=ldq)
    return _lib.swiglu_quant_s8(type, T, N, gate, ldg, up, ldu, q, ldq, scale, stream)


def swiglu_quant_f8(type, T, N, gate, ldg, up, ldu, q, ldq, scale, lds, stream=0) -> int:
    _int32(type=type, T=T, N=N, ldg=ldg, ldu=ldu, ldq=ldq, lds=lds)
    return _lib.swiglu_quant_f8(type, T, N, gate, ldg, up, ldu, q, ldq, scale, lds, stream)


# The wrappers below are called for single tokens, where their own time is what
# counts.  Calls with dense tensors on the current device and no stream named go
# through _calls (csrc/calls.cpp), which checks the same things natively; it
# returns None for all others, which the Python below makes or refuses.
if _calls is not None:
    _calls.bind(TDI8Error, *(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in (
        "rmsnorm_quant_s8", "rmsnorm_quant_f8", "swiglu_quant_s8", "swiglu_quant_f8", "gemm_s8s8_grouped",
        "gemm_f8f8_block128")))
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(index: int, fn, args, stream) -> None:
    """fn(*args, stream handle) with device `index` current; raises TDI8Error."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(index, fn, args, stream)
    st = fn(*args, _current_stream(index) if stream is None else _stream_handle(stream))
    if st != OK:
        raise TDI8Error(st)


def _gpu(*tensors) -> int:
    """Index of the one GPU holding every tensor (None skipped)."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != index or index < 0):
            _device_of(*(t for t in tensors if t is not None))  # says what is wrong
            raise ValueError("tensors must be on one GPU")
    return index


def _fit(*values) -> None:
    if max(values) > INT_MAX:
        raise ValueError(f"a size or stride of {max(values)} does not fit the library's int arguments (< 2**31)")


def _stored(name, t) -> None:
    """Refuses a tensor whose memory holds something else than its values."""
    if t.is_neg():
        raise ValueError(f"{name} is negated lazily: pass its resolve_neg()")


def _matrix(name, t, dtype, shape=None) -> int:
    """Checks a 2-D tensor with unit column stride; its leading dimension."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    _stored(name, t)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, cols = size = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(size)}")
    if rows > 1:
        if ld < cols:
            raise ValueError(f"{name}'s rows overlap")
        return ld
    return cols if cols > 1 else 1


def _empty(like, shape, dtype, stream):
    """A new tensor of the stream that the call runs on (so that its memory
    is not handed out again while the call still runs)."""
    if stream is None:
        if like.shape == shape and like.is_contiguous():
            return torch.empty_like(like, dtype=dtype)  # the cheapest of torch's ways
        return like.new_empty(shape, dtype=dtype)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _eight_bit_out(fmt, T, H, like, out, scale, stream):
    """The 8-bit output and its scales, the caller's, checked, or new ones, and their leading dimensions."""
    if fmt == "s8":
        dtype, shape = torch.int8, (T,)
    elif fmt == "f8":
        dtype, shape = torch.float8_e4m3fn, (T, (H + BLOCK - 1) // BLOCK)
    else:
        raise ValueError(f"fmt must be 's8' or 'f8', not {fmt!r}")
    if out is None:
        out, ldq = _empty(like, (T, H), dtype, stream), max(H, 1)
    else:
        ldq = _matrix("out", out, dtype, (T, H))
    lds = max(shape[-1], 1)
    if scale is None:
        scale = _empty(like, shape, torch.float32, stream)
    elif fmt == "f8":
        lds = _matrix("scale", scale, torch.float32, shape)
    else:
        _vector("scale", scale, torch.float32, T)
    return out, ldq, scale, lds


def _outputs(**given) -> None:
    """Refuses outputs that autograd would take for what they were: results carry no gradients."""
    for name, t in given.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires grad, and results carry no gradients: write to it under torch.no_grad()")


def _written(*given) -> None:
    """The caller's outputs count as written, for backward passes that kept them."""
    for t in given:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _vector(name, t, dtype, count) -> None:
    if t.dtype != dtype or t.shape != (count,) or (count > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a dense {dtype} vector of {count} values")
    _stored(name, t)


def rms_norm(x, weight, eps: float = 1e-6, residual=None, fmt: str = "s8", sum_out=None, out=None, scale=None,
             stream=None):
    """RMS norm of x (T, H) with an 8-bit output: (q, scale), or with a
    residual (q, scale, sum) for the norm of sum = x + residual.

    x, residual, weight (H): float32, bfloat16 or float16, all alike, with
       unit column stride.
    fmt: "s8": q int8 with scale (T); "f8": q float8_e4m3fn with scale
       (T, ceil(H / 128)), one for each block of 128 columns.
    sum_out: where the sum goes (x or residual itself: in place).

    Results carry no gradients, also where inputs require them; sum_out, out
    and scale count as written in place for tensors that a backward pass kept.
    """
    if _calls is not None and stream is None and x.is_cuda:
        device = _current_device()
        made = _calls.rms_norm(x, weight, eps, residual, fmt, sum_out, out, scale, device, _current_stream(device))
        if made is not None:
            return made
    _outputs(sum_out=sum_out, out=out, scale=scale)
    given = sum_out, out, scale
    dtype = x.dtype
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    ldx = _matrix("x", x, dtype)
    T, H = shape = x.shape
    _vector("weight", weight, dtype, H)
    ldr = ldsum = 0
    if residual is not None:
        ldr = _matrix("residual", residual, dtype, shape)
        if sum_out is not None:
            ldsum = _matrix("sum_out", sum_out, dtype, shape)
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    index = _gpu(x, weight, residual, sum_out, out, scale)
    if residual is not None and sum_out is None:
        sum_out, ldsum = _empty(x, shape, dtype, stream), max(H, 1)
    out, ldq, scale, lds = _eight_bit_out(fmt, T, H, x, out, scale, stream)
    _fit(T, H, ldx, ldr, ldsum, ldq, lds)
    args = (code, T, H, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, weight.data_ptr(),
            eps, None if residual is None else sum_out.data_ptr(), ldsum, out.data_ptr(), ldq, scale.data_ptr())
    if fmt == "s8":
        _call(index, _lib.rmsnorm_quant_s8, args, stream)
    else:
        _call(index, _lib.rmsnorm_quant_f8, args + (lds,), stream)
    _written(*given)
    return (out, scale) if residual is None else (out, scale, sum_out)


def swiglu(gate, up, fmt: str = "s8", out=None, scale=None, stream=None):
    """(q, scale) of gate / (1 + exp(-gate)) * up for gate and up (T, N), in
    the formats of rms_norm; the two may be halves of one tensor's rows.
    Gradients as for rms_norm."""
    if _calls is not None and stream is None and gate.is_cuda:
        device = _current_device()
        made = _calls.swiglu(gate, up, fmt, out, scale, device, _current_stream(device))
        if made is not None:
            return made
    _outputs(out=out, scale=scale)
    given = out, scale
    dtype = gate.dtype
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError("gate must be float32, bfloat16 or float16")
    ldg = _matrix("gate", gate, dtype)
    T, N = shape = gate.shape
    ldu = _matrix("up", up, dtype, shape)
    index = _gpu(gate, up, out, scale)
    out, ldq, scale, lds = _eight_bit_out(fmt, T, N, gate, out, scale, stream)
    _fit(T, N, ldg, ldu, ldq, lds)
    args = (code, T, N, gate.data_ptr(), ldg, up.data_ptr(), ldu, out.data_ptr(), ldq, scale.data_ptr())
    if fmt == "s8":
        _call(index, _lib.swiglu_quant_s8, args, stream)
    else:
        _call(index, _lib.swiglu_quant_f8, args + (lds,), stream)
    _written(*given)
    return out, scale


# ---- products of 8-bit operands with their scales -------------------------------------

def gemm_s8s8_grouped(type, G, M, N, K, A, lda, a_rows, a_scale, rows, offsets, B, ldb, group_b, b_scale, C, ldc,
                      stream=0) -> int:
    _int32(type=type, G=G, M=M, N=N, K=K, lda=lda, a_rows=a_rows, ldb=ldb, ldc=ldc)
    if not -2 ** 63 <= int(group_b) < 2 ** 63:
        raise ValueError(f"group_b = {group_b} does not fit the library's 64-bit argument")
    return _lib.gemm_s8s8_grouped(type, G, M, N, K, A, lda, a_rows, a_scale, rows, offsets, B, ldb, group_b, b_scale,
                                  C, ldc, stream)


def gemm_f8f8_block128(type, M, N, K, A, lda, a_scale, ldas, B, ldb, b_scale, ldbs, C, ldc, stream=0) -> int:
    _int32(type=type, M=M, N=N, K=K, lda=lda, ldas=ldas, ldb=ldb, ldbs=ldbs, ldc=ldc)
    return _lib.gemm_f8f8_block128(type, M, N, K, A, lda, a_scale, ldas, B, ldb, b_scale, ldbs, C, ldc, stream)


def scaled_product_plan(f8, type, G, M, N, K, aligned, num_cu) -> ScaledPlan:
    """What the scaled product of these sizes would enqueue; raises TDI8Error for sizes it refuses."""
    _int32(type=type, G=G, M=M, N=N, K=K, num_cu=num_cu)
    out = ScaledPlan()
    st = _lib.scaled_product_plan(1 if f8 else 0, type, G, M, N, K, 1 if aligned else 0, num_cu, ctypes.byref(out))
    if st != OK:
        raise TDI8Error(st)
    return out


def _product_out(M, N, dtype, like, out, stream):
    """The product's output, the caller's, checked, or a new one, and its leading dimension."""
    if out is None:
        if dtype not in _TYPES:
            raise TypeError("dtype must be float32, bfloat16 or float16")
        return _empty(like, (M, N), dtype, stream), max(N, 1)
    if out.dtype not in _TYPES:
        raise TypeError("out must be float32, bfloat16 or float16")
    return out, _matrix("out", out, out.dtype, (M, N))


def grouped_gemm(A, a_scale, B, b_scale, offsets=None, rows=None, out=None, dtype=torch.bfloat16, stream=None):
    """int8 products grouped by expert, with their scales: row r of the
    result, in group g (offsets[g] <= r < offsets[g + 1]), is
    a_scale[i] * b_scale[g] * (A[i] x B[g] transposed) with i = rows[r] or r.

    A: int8 (T, K); a_scale: float32 (T), as rms_norm and swiglu give them.
    B: int8 (G, N, K) with b_scale float32 (G, N), or (N, K) with (N).  Groups
       and rows may lie apart but not overlap (no weights shared by a zero
       stride).
    offsets: int32 (G + 1) on the GPU (not needed for one group of all rows).
    rows: int32 row indices into A, one for each row of the result (rows
       outside A give zeros, but A has one row at least); without them the
       result has A's rows.
    out: (M, N) of a floating type, or dtype for a new tensor; rows from
       offsets[G] on are not written.

    Gradients as for rms_norm.
    """
    if _calls is not None and stream is None and A.is_cuda:
        device = _current_device()
        made = _calls.grouped_gemm(A, a_scale, B, b_scale, offsets, rows, out, dtype, device, _current_stream(device))
        if made is not None:
            return made
    _outputs(out=out)
    given = out
    lda = _matrix("A", A, torch.int8)
    T, K = A.shape
    if B.dtype != torch.int8:
        raise TypeError(f"B must be torch.int8, not {B.dtype}")
    _stored("B", B)
    _stored("b_scale", b_scale)
    if B.dim() == 2:
        B, b_scale = B[None], b_scale[None]
    if B.dim() != 3 or B.shape[2] != K or (K > 1 and B.stride(2) != 1):
        raise ValueError("B must be (G, N, K) or (N, K) with A's K and unit stride along it")
    G, N, _ = B.shape
    if b_scale.dtype != torch.float32 or b_scale.shape != (G, N) or not b_scale.is_contiguous():
        raise ValueError(f"b_scale must be a dense float32 tensor of shape {(G, N)}")
    _vector("a_scale", a_scale, torch.float32, T)
    if offsets is not None:
        _vector("offsets", offsets, torch.int32, G + 1)
    elif G != 1:
        raise ValueError("offsets are needed for more than one group")
    M = T
    if rows is not None:
        M = rows.numel()
        _vector("rows", rows, torch.int32, M)
    ldb = B.stride(1) if N > 1 else max(K, 1)
    if M > 0 and N > 0 and G > 0:
        if T == 0:
            raise ValueError("A has no rows for `rows` to name")
        if ldb < K:
            raise ValueError("B's rows overlap")
        if G > 1 and B.stride(0) < (N - 1) * ldb + K:
            raise ValueError("B's groups overlap: weights that groups share need a copy for each")
    index = _gpu(A, a_scale, B, b_scale, offsets, rows, out)
    out, ldc = _product_out(M, N, dtype, A, out, stream)
    _fit(G, M, N, K, lda, T, ldb, ldc)
    _call(index, _lib.gemm_s8s8_grouped,
          (_TYPES[out.dtype], G, M, N, K, A.data_ptr(), lda, T, a_scale.data_ptr(),
           None if rows is None else rows.data_ptr(), None if offsets is None else offsets.data_ptr(), B.data_ptr(),
           ldb, B.stride(0) if G > 1 else 0, b_scale.data_ptr(), out.data_ptr(), ldc), stream)
    _written(given)
    return out


def gemm_f8(A, a_scale, B, b_scale, out=None, dtype=torch.bfloat16, stream=None):
    """A x B transposed for e4m3 operands with a scale for each block of 128.

    A: float8_e4m3fn (M, K), a_scale: float32 (M, ceil(K / 128)), as rms_norm
       and swiglu give them with fmt="f8".
    B: float8_e4m3fn (N, K), b_scale: float32 (ceil(N / 128), ceil(K / 128)).
    out: (M, N) of a floating type, or dtype for a new tensor.  float32 and
       float16 hold all sums in 32 bits; bfloat16 takes the e4m3 matrix
       instructions' sums, in which of 8 consecutive products those below
       2^-13 of the largest are lost, at twice the rate.

    Gradients as for rms_norm.
    """
    if _calls is not None and stream is None and A.is_cuda:
        device = _current_device()
        made = _calls.gemm_f8(A, a_scale, B, b_scale, out, dtype, device, _current_stream(device))
        if made is not None:
            return made
    _outputs(out=out)
    given = out
    lda = _matrix("A", A, torch.float8_e4m3fn)
    ldb = _matrix("B", B, torch.float8_e4m3fn)
    (M, K), N = A.shape, B.shape[0]
    if B.shape[1] != K:
        raise ValueError("inner dimensions differ")
    kb = (K + BLOCK - 1) // BLOCK
    ldas = _matrix("a_scale", a_scale, torch.float32, (M, kb))
    ldbs = _matrix("b_scale", b_scale, torch.float32, ((N + BLOCK - 1) // BLOCK, kb))
    index = _gpu(A, a_scale, B, b_scale, out)
    out, ldc = _product_out(M, N, dtype, A, out, stream)
    _fit(M, N, K, lda, ldas, ldb, ldbs, ldc)
    _call(index, _lib.gemm_f8f8_block128,
          (_TYPES[out.dtype], M, N, K, A.data_ptr(), lda, a_scale.data_ptr(), ldas, B.data_ptr(), ldb,
           b_scale.data_ptr(), ldbs, out.data_ptr(), ldc), stream)
    _written(given)
    return out
