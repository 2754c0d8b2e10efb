"""Python binding of the C ABI in ``include/tcq.h`` (argument marshalling only).

The functions named like the C entry points (``tcq_encode`` ...) take raw device
pointers and sizes exactly as the C ABI does.  ``encode``/``decode`` accept
torch CUDA tensors, allocate outputs and workspace with torch, and launch on the
current torch stream; ``encode_host`` additionally stages host arrays through
pinned memory (the end-to-end path).  Every step of the search and the decode
runs in the CUDA library: when it is missing this module raises instead of
computing anything itself.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
# TCQ_LIBRARY=debug selects the bounds-checked build (libtcq_debug.so, see
# build.py); load only one of the two builds in a process.
LIB_PATH = os.path.join(_PKG, "libtcq_debug.so" if os.environ.get("TCQ_LIBRARY") == "debug"
                        else "libtcq.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "tcq.h")

TCQ_OK = 0
TCQ_ERR_INVALID_ARG = 1
TCQ_ERR_UNSUPPORTED = 2
TCQ_ERR_WORKSPACE = 3
TCQ_ERR_CUDA = 4
TCQ_ERR_INTERNAL = 5
TCQ_F32 = 0
TCQ_F16 = 1
TCQ_MAD = 2
TCQ_X_F16 = 0
TCQ_X_BF16 = 1
TCQ_ACT_NONE = 0
TCQ_ACT_RELU = 1
TCQ_ACT_SILU = 2
TCQ_ACT_GELU = 3
TCQ_ACT_GELU_TANH = 4
TCQ_Q8_INT8 = 0
TCQ_Q8_E4M3 = 1
ACTIVATIONS = {"none": TCQ_ACT_NONE, "relu": TCQ_ACT_RELU, "silu": TCQ_ACT_SILU, "gelu": TCQ_ACT_GELU,
               "gelu_tanh": TCQ_ACT_GELU_TANH}
Q8_FORMATS = {"int8": TCQ_Q8_INT8, "e4m3": TCQ_Q8_E4M3}


class _ComputedCode:
    """Stands for the computed (lookup-free) code wherever a codebook tensor goes."""

    def __repr__(self):
        return "MAD"


MAD = _ComputedCode()  # pass as ``codebook`` to select TCQ_MAD
TCQ_MAX_L = 16
TCQ_MAX_K = 4
TCQ_MAX_T = 1 << 20

_lib = None


class TCQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {tcq_status_string(status)}")


def load_library() -> ctypes.CDLL:
    """Load ``libtcq.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m trellis_coded_weight_tcq_b200.build` "
            "(there is no CPU fallback)"
        )
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i64, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
    lib.tcq_words_per_block.argtypes = [ci, ci]
    lib.tcq_words_per_block.restype = ci
    lib.tcq_encode_workspace_bytes.argtypes = [ci, ci, ci, i64, ci]
    lib.tcq_encode_workspace_bytes.restype = sz
    lib.tcq_encode.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp, vp, vp, sz, vp]
    lib.tcq_encode.restype = ci
    lib.tcq_encode_fixed_start.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp, vp, vp, vp,
                                           sz, vp]
    lib.tcq_encode_fixed_start.restype = ci
    lib.tcq_encode_vec_workspace_bytes.argtypes = [ci, ci, ci, ci, i64, ci]
    lib.tcq_encode_vec_workspace_bytes.restype = sz
    lib.tcq_encode_vec.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, i64, vp, vp, vp, vp, sz, vp]
    lib.tcq_encode_vec.restype = ci
    lib.tcq_decode_vec.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, i64, vp, vp]
    lib.tcq_decode_vec.restype = ci
    lib.tcq_decode.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp]
    lib.tcq_decode.restype = ci
    lib.tcq_status_string.argtypes = [ci]
    lib.tcq_status_string.restype = ctypes.c_char_p
    lib.tcq_encode_path.argtypes = [ci, ci, ci]
    lib.tcq_encode_path.restype = ctypes.c_char_p
    lib.tcq_gemv.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, i64, i64, vp, vp, vp]
    lib.tcq_gemv.restype = ci
    lib.tcq_gemv_vec.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, i64, i64, vp, vp, vp]
    lib.tcq_gemv_vec.restype = ci
    lib.tcq_ldlq_workspace_bytes.argtypes = [ci, ci, ci, i64, i64, ci]
    lib.tcq_ldlq_workspace_bytes.restype = sz
    lib.tcq_ldlq.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, i64, i64, vp, vp, vp, vp, vp, vp,
                             sz, vp]
    lib.tcq_ldlq.restype = ci
    lib.tcq_bcjr_workspace_bytes.argtypes = [ci, ci, ci, i64, ci]
    lib.tcq_bcjr_workspace_bytes.restype = sz
    lib.tcq_bcjr.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.tcq_bcjr.restype = ci
    lib.tcq_ub8_words_per_block.argtypes = [ci, ci, ci]
    lib.tcq_ub8_words_per_block.restype = ci
    lib.tcq_ub8_encode.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp, vp, vp, vp]
    lib.tcq_ub8_encode.restype = ci
    lib.tcq_ub8_decode.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp]
    lib.tcq_ub8_decode.restype = ci
    lib.tcq_pack8.argtypes = [vp, ci, i64, i64, i64, ci, vp, vp, vp]
    lib.tcq_pack8.restype = ci
    lib.tcq_unpack8.argtypes = [vp, vp, ci, i64, i64, vp, ci, i64, vp]
    lib.tcq_unpack8.restype = ci
    lib.tcq_gemm_workspace_bytes.argtypes = [ci, ci, ci, i64, i64, i64, ci]
    lib.tcq_gemm_workspace_bytes.restype = sz
    lib.tcq_gemm.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, i64, i64, vp, ci, i64, i64, vp, ci, vp, i64, vp, i64,
                             vp, vp, ci, vp, sz, vp]
    lib.tcq_gemm.restype = ci
    lib.tcq_gemm_dgrad_workspace_bytes.argtypes = [ci, ci, ci, i64, i64, i64, ci]
    lib.tcq_gemm_dgrad_workspace_bytes.restype = sz
    lib.tcq_gemm_dgrad.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, i64, i64, vp, ci, i64, i64, vp, i64, vp, sz, vp]
    lib.tcq_gemm_dgrad.restype = ci
    lib.tcq_act_grad8_workspace_bytes.argtypes = [i64, i64]
    lib.tcq_act_grad8_workspace_bytes.restype = sz
    lib.tcq_act_grad8.argtypes = [vp, ci, i64, vp, vp, ci, ci, i64, i64, vp, i64, vp, vp, sz, vp]
    lib.tcq_act_grad8.restype = ci
    lib.tcq_wgrad8_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tcq_wgrad8_workspace_bytes.restype = sz
    lib.tcq_wgrad8.argtypes = [vp, ci, i64, vp, vp, ci, i64, i64, i64, vp, i64, ci, vp, sz, vp]
    lib.tcq_wgrad8.restype = ci
    lib.tcq_device_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.tcq_device_errors.restype = ci
    _lib = lib
    return lib


def header_functions() -> list[str]:
    """Names of the functions ``include/tcq.h`` declares."""
    with open(HEADER_PATH) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(tcq_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------------------
# the C entry points, one to one
# ---------------------------------------------------------------------------
def tcq_words_per_block(k: int, T: int) -> int:
    return int(load_library().tcq_words_per_block(k, T))


def tcq_encode_workspace_bytes(L: int, k: int, T: int, n_blocks: int, cb_dtype: int) -> int:
    return int(load_library().tcq_encode_workspace_bytes(L, k, T, n_blocks, cb_dtype))


def tcq_encode(x, d, codebook, cb_dtype, L, k, T, n_blocks, start_state, bits, path_cost,
               workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_encode(x, d, codebook, cb_dtype, L, k, T, n_blocks, start_state,
                                          bits, path_cost, workspace, workspace_bytes, stream))


def tcq_encode_fixed_start(x, d, codebook, cb_dtype, L, k, T, n_blocks, fixed_start, start_state,
                           bits, path_cost, workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_encode_fixed_start(x, d, codebook, cb_dtype, L, k, T, n_blocks,
                                                     fixed_start, start_state, bits, path_cost,
                                                     workspace, workspace_bytes, stream))


def tcq_encode_vec_workspace_bytes(L, k, V, T, n_blocks, cb_dtype) -> int:
    return int(load_library().tcq_encode_vec_workspace_bytes(L, k, V, T, n_blocks, cb_dtype))


def tcq_encode_vec(x, d, codebook, cb_dtype, L, k, V, T, n_blocks, start_state, bits, path_cost,
                   workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_encode_vec(x, d, codebook, cb_dtype, L, k, V, T, n_blocks,
                                             start_state, bits, path_cost, workspace,
                                             workspace_bytes, stream))


def tcq_decode_vec(bits, start_state, codebook, cb_dtype, L, k, V, T, n_blocks, y, stream) -> int:
    return int(load_library().tcq_decode_vec(bits, start_state, codebook, cb_dtype, L, k, V, T,
                                             n_blocks, y, stream))


def tcq_decode(bits, start_state, codebook, cb_dtype, L, k, T, n_blocks, y, stream) -> int:
    return int(load_library().tcq_decode(bits, start_state, codebook, cb_dtype, L, k, T, n_blocks,
                                          y, stream))


def tcq_gemv(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols, x, y, stream) -> int:
    return int(load_library().tcq_gemv(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows,
                                        cols, x, y, stream))


def tcq_gemv_vec(bits, start_state, scale, codebook, cb_dtype, L, k, V, T, rows, cols, x, y,
                 stream) -> int:
    return int(load_library().tcq_gemv_vec(bits, start_state, scale, codebook, cb_dtype, L, k, V, T,
                                            rows, cols, x, y, stream))


def tcq_ldlq_workspace_bytes(L: int, k: int, T: int, rows: int, cols: int, cb_dtype: int) -> int:
    return int(load_library().tcq_ldlq_workspace_bytes(L, k, T, rows, cols, cb_dtype))


def tcq_ldlq(w, u, d, codebook, cb_dtype, L, k, T, rows, cols, q, x, start_state, bits, path_cost,
             workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_ldlq(w, u, d, codebook, cb_dtype, L, k, T, rows, cols, q, x,
                                       start_state, bits, path_cost, workspace, workspace_bytes,
                                       stream))


def tcq_bcjr_workspace_bytes(L: int, k: int, T: int, n_blocks: int, cb_dtype: int) -> int:
    return int(load_library().tcq_bcjr_workspace_bytes(L, k, T, n_blocks, cb_dtype))


def tcq_bcjr(x, d, codebook, cb_dtype, L, k, T, n_blocks, tau, y_soft, free_energy, workspace,
             workspace_bytes, stream) -> int:
    return int(load_library().tcq_bcjr(x, d, codebook, cb_dtype, L, k, T, n_blocks, tau, y_soft,
                                       free_energy, workspace, workspace_bytes, stream))


def tcq_ub8_words_per_block(V: int, m: int, T: int) -> int:
    return int(load_library().tcq_ub8_words_per_block(V, m, T))


def tcq_ub8_encode(x, d, codebook, cb_dtype, V, m, T, n_blocks, fixed_start, start_state, bits,
                   path_cost, stream) -> int:
    return int(load_library().tcq_ub8_encode(x, d, codebook, cb_dtype, V, m, T, n_blocks,
                                             fixed_start, start_state, bits, path_cost, stream))


def tcq_ub8_decode(bits, start_state, codebook, cb_dtype, V, m, T, n_blocks, y, stream) -> int:
    return int(load_library().tcq_ub8_decode(bits, start_state, codebook, cb_dtype, V, m, T,
                                             n_blocks, y, stream))


def tcq_pack8(x, xdtype, ldx, n, cols, fmt, codes, scales, stream) -> int:
    return int(load_library().tcq_pack8(x, xdtype, ldx, n, cols, fmt, codes, scales, stream))


def tcq_unpack8(codes, scales, fmt, n, cols, x, xdtype, ldx, stream) -> int:
    return int(load_library().tcq_unpack8(codes, scales, fmt, n, cols, x, xdtype, ldx, stream))


def tcq_gemm_workspace_bytes(L, k, T, rows, cols, n, cb_dtype) -> int:
    return int(load_library().tcq_gemm_workspace_bytes(L, k, T, rows, cols, n, cb_dtype))


def tcq_gemm(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols, x, xdtype, ldx, n, bias, act,
             residual, ldr, y, ldy, z_codes, z_scales, z_format, workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_gemm(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols, x, xdtype,
                                       ldx, n, bias, act, residual, ldr, y, ldy, z_codes, z_scales, z_format,
                                       workspace, workspace_bytes, stream))


def tcq_gemm_dgrad_workspace_bytes(L, k, T, rows, cols, n, cb_dtype) -> int:
    return int(load_library().tcq_gemm_dgrad_workspace_bytes(L, k, T, rows, cols, n, cb_dtype))


def tcq_gemm_dgrad(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols, dz, xdtype, lddz, n, dx, lddx,
                   workspace, workspace_bytes, stream) -> int:
    return int(load_library().tcq_gemm_dgrad(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols, dz,
                                             xdtype, lddz, n, dx, lddx, workspace, workspace_bytes, stream))


def tcq_act_grad8_workspace_bytes(n: int, rows: int) -> int:
    return int(load_library().tcq_act_grad8_workspace_bytes(n, rows))


def tcq_act_grad8(dy, xdtype, lddy, z_codes, z_scales, z_format, act, n, rows, dz, lddz, dbias, workspace,
                  workspace_bytes, stream) -> int:
    return int(load_library().tcq_act_grad8(dy, xdtype, lddy, z_codes, z_scales, z_format, act, n, rows, dz, lddz,
                                            dbias, workspace, workspace_bytes, stream))


def tcq_wgrad8_workspace_bytes(rows: int, cols: int, n: int) -> int:
    return int(load_library().tcq_wgrad8_workspace_bytes(rows, cols, n))


def tcq_wgrad8(dz, xdtype, lddz, x_codes, x_scales, x_format, n, rows, cols, dw, lddw, accumulate, workspace,
               workspace_bytes, stream) -> int:
    return int(load_library().tcq_wgrad8(dz, xdtype, lddz, x_codes, x_scales, x_format, n, rows, cols, dw, lddw,
                                         accumulate, workspace, workspace_bytes, stream))


TCQ_DEVERR_WAIT_TIMEOUT = 0x1
TCQ_DEVERR_BOUNDS = 0x2


def tcq_device_errors(stream, flags) -> int:
    return int(load_library().tcq_device_errors(stream, flags))


def device_errors(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error flags."""
    flags = ctypes.c_uint32(0)
    st = tcq_device_errors(_stream_handle(stream), ctypes.byref(flags))
    if st not in (TCQ_OK, TCQ_ERR_INTERNAL):
        raise TCQError(st, "tcq_device_errors")
    return int(flags.value)


def tcq_status_string(status: int) -> str:
    return load_library().tcq_status_string(status).decode()


def tcq_encode_path(L: int, k: int, cb_dtype: int) -> str:
    return load_library().tcq_encode_path(L, k, cb_dtype).decode()


# ---------------------------------------------------------------------------
# torch conveniences (device memory and streams only)
# ---------------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def cb_dtype_of(codebook) -> int:
    if codebook is MAD:
        return TCQ_MAD
    torch = _torch()
    if codebook.dtype == torch.float16:
        return TCQ_F16
    if codebook.dtype == torch.float32:
        return TCQ_F32
    raise TypeError(f"codebook must be float16 or float32, got {codebook.dtype}")


def _ptr(t):
    return None if t is None or t is MAD else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, what: str) -> None:
    if status != TCQ_OK:
        raise TCQError(status, what)


@dataclass
class Encoded:
    start_state: "object"  # uint32 [n] as torch.int32 storage
    bits: "object"         # uint32 [n, W] as torch.int32 storage
    path_cost: "object"    # float32 [n]


class Workspace:
    """A reusable device workspace for ``encode`` (torch-allocated)."""

    def __init__(self, L: int, k: int, T: int, n_blocks: int, cb_dtype: int, device=None):
        torch = _torch()
        self.nbytes = max(tcq_encode_workspace_bytes(L, k, T, n_blocks, cb_dtype), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")


def encode(x, d, codebook, L: int, k: int, workspace: Workspace | None = None, out=None,
           stream=None, fixed_start=None) -> Encoded:
    """Viterbi TCQ of every row of ``x`` (fp32 CUDA tensor [n_blocks, T]); a free
    start state per block, or the int32 tensor ``fixed_start`` of start states."""
    torch = _torch()
    if x.dim() != 2 or x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor [n_blocks, T]")
    n, T = x.shape
    if d is not None and (d.shape != x.shape or d.dtype != torch.float32 or not d.is_contiguous()):
        raise ValueError("d must be None or a contiguous float32 tensor shaped like x")
    W = tcq_words_per_block(k, T)
    if W < 0:
        raise TCQError(TCQ_ERR_UNSUPPORTED, "tcq_words_per_block")
    if out is None:
        out = Encoded(
            torch.empty(n, dtype=torch.int32, device=x.device),
            torch.empty((n, W), dtype=torch.int32, device=x.device),
            torch.empty(n, dtype=torch.float32, device=x.device),
        )
    ws = workspace or Workspace(L, k, T, n, cb_dtype_of(codebook), x.device)
    if fixed_start is None:
        _check(tcq_encode(_ptr(x), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), L, k, T, n,
                          _ptr(out.start_state), _ptr(out.bits), _ptr(out.path_cost),
                          ctypes.c_void_p(ws.buf.data_ptr()), ws.nbytes, _stream_handle(stream)),
               "tcq_encode")
    else:
        if fixed_start.numel() < n or fixed_start.dtype != torch.int32 or not fixed_start.is_cuda:
            raise ValueError("fixed_start must be an int32 CUDA tensor of n_blocks start states")
        _check(tcq_encode_fixed_start(_ptr(x), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), L,
                                      k, T, n, _ptr(fixed_start), _ptr(out.start_state),
                                      _ptr(out.bits), _ptr(out.path_cost),
                                      ctypes.c_void_p(ws.buf.data_ptr()), ws.nbytes,
                                      _stream_handle(stream)), "tcq_encode_fixed_start")
    return out


def decode(bits, start_state, codebook, L: int, k: int, T: int, out=None, stream=None):
    """Values [n_blocks, T] (fp32) of packed ``bits`` from ``start_state``."""
    torch = _torch()
    n = start_state.shape[0]
    W = tcq_words_per_block(k, T)
    if bits.numel() < n * max(W, 0):
        raise ValueError("decode: bits holds fewer than n_blocks * W words")
    if out is None:
        out = torch.empty((n, T), dtype=torch.float32, device=bits.device)
    if out.numel() < n * T:
        raise ValueError("decode: out holds fewer than n_blocks * T values")
    _check(tcq_decode(_ptr(bits), _ptr(start_state), _ptr(codebook), cb_dtype_of(codebook), L, k,
                      T, n, _ptr(out), _stream_handle(stream)), "tcq_decode")
    return out


def gemv(bits, start_state, scale, codebook, L: int, k: int, T: int, rows: int, cols: int, x,
         out=None, stream=None):
    """y = (trellis-coded matrix) @ x, decoding on the fly; blocks row-major [rows, cols/T]."""
    torch = _torch()
    nb = rows * (cols // T) if T > 0 else 0
    W = tcq_words_per_block(k, T)
    if bits.numel() < nb * max(W, 0) or start_state.numel() < nb or x.numel() < cols or (
            scale is not None and scale.numel() < nb):
        raise ValueError(f"gemv: tensors too small for a {rows} x {cols} matrix of T={T} blocks")
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=x.device)
    if out.numel() < rows:
        raise ValueError("gemv: out holds fewer than rows values")
    _check(tcq_gemv(_ptr(bits), _ptr(start_state), _ptr(scale), _ptr(codebook),
                    cb_dtype_of(codebook), L, k, T, rows, cols, _ptr(x), _ptr(out),
                    _stream_handle(stream)), "tcq_gemv")
    return out


def gemv_vec(bits, start_state, scale, codebook, L: int, k: int, V: int, T: int, rows: int,
             cols: int, x, out=None, stream=None):
    """gemv for the vector trellis (V weights per step, codebook [2^L, V])."""
    torch = _torch()
    nb = rows * (cols // T) if T > 0 else 0
    W = tcq_words_per_block(k, T)
    if bits.numel() < nb * max(W, 0) or start_state.numel() < nb or x.numel() < cols or (
            scale is not None and scale.numel() < nb):
        raise ValueError(f"gemv_vec: tensors too small for a {rows} x {cols} matrix of T={T} blocks")
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=x.device)
    if out.numel() < rows:
        raise ValueError("gemv_vec: out holds fewer than rows values")
    _check(tcq_gemv_vec(_ptr(bits), _ptr(start_state), _ptr(scale), _ptr(codebook),
                        cb_dtype_of(codebook), L, k, V, T, rows, cols, _ptr(x), _ptr(out),
                        _stream_handle(stream)), "tcq_gemv_vec")
    return out


@dataclass
class LdlqResult:
    q: "object"            # float32 [rows, cols], the reconstruction
    x: "object"            # float32 [rows, cols], the targets, or None
    coded: Encoded         # blocks (r, j) at r * (cols / T) + j


def ldlq(w, u, d, codebook, L: int, k: int, T: int, keep_targets: bool = True, workspace=None,
         stream=None) -> LdlqResult:
    """Error-feedback TCQ of the matrix ``w`` (fp32 CUDA [rows, cols]) by column
    blocks of T, with H = U diag(d) U^T (``u`` fp32 [cols, cols], ``d`` fp32 [cols]
    or None)."""
    torch = _torch()
    if w.dim() != 2 or w.dtype != torch.float32 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous float32 CUDA tensor [rows, cols]")
    rows, cols = w.shape
    if u.shape != (cols, cols) or u.dtype != torch.float32 or not u.is_contiguous():
        raise ValueError("u must be a contiguous float32 tensor [cols, cols]")
    if d is not None and (d.shape != (cols,) or d.dtype != torch.float32 or not d.is_contiguous()):
        raise ValueError("d must be None or a contiguous float32 tensor [cols]")
    W = tcq_words_per_block(k, T)
    if W < 0:
        raise TCQError(TCQ_ERR_UNSUPPORTED, "tcq_words_per_block")
    nb = cols // T if T > 0 else 0
    dev = w.device
    q = torch.empty((rows, cols), dtype=torch.float32, device=dev)
    x = torch.empty((rows, cols), dtype=torch.float32, device=dev) if keep_targets else None
    coded = Encoded(
        torch.empty(rows * nb, dtype=torch.int32, device=dev),
        torch.empty((rows * nb, W), dtype=torch.int32, device=dev),
        torch.empty(rows * nb, dtype=torch.float32, device=dev),
    )
    if workspace is None:
        nbytes = max(tcq_ldlq_workspace_bytes(L, k, T, rows, cols, cb_dtype_of(codebook)), 256)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(tcq_ldlq(_ptr(w), _ptr(u), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), L, k, T,
                    rows, cols, _ptr(q), _ptr(x), _ptr(coded.start_state), _ptr(coded.bits),
                    _ptr(coded.path_cost), ctypes.c_void_p(workspace.data_ptr()),
                    workspace.numel(), _stream_handle(stream)), "tcq_ldlq")
    return LdlqResult(q, x, coded)


def bcjr(x, d, codebook, L: int, k: int, tau: float, workspace=None, out=None, stream=None):
    """Soft codewords [n_blocks, T] and free energies -tau ln Z [n_blocks] of the
    rows of ``x`` (fp32 CUDA [n_blocks, T]) at temperature ``tau``."""
    torch = _torch()
    if x.dim() != 2 or x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor [n_blocks, T]")
    n, T = x.shape
    if d is not None and (d.shape != x.shape or d.dtype != torch.float32 or not d.is_contiguous()):
        raise ValueError("d must be None or a contiguous float32 tensor shaped like x")
    if out is None:
        out = (torch.empty((n, T), dtype=torch.float32, device=x.device),
               torch.empty(n, dtype=torch.float32, device=x.device))
    y, F = out
    if y.numel() < n * T or (F is not None and F.numel() < n):
        raise ValueError("bcjr: output tensors too small")
    if workspace is None:
        nbytes = max(tcq_bcjr_workspace_bytes(L, k, T, n, cb_dtype_of(codebook)), 256)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _check(tcq_bcjr(_ptr(x), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), L, k, T, n,
                    float(tau), _ptr(y), _ptr(F), ctypes.c_void_p(workspace.data_ptr()),
                    workspace.numel(), _stream_handle(stream)), "tcq_bcjr")
    return y, F


def encode_vec(x, d, codebook, L: int, k: int, V: int, workspace=None, out=None,
               stream=None) -> Encoded:
    """Viterbi TCQ over the vector trellis: V weights per step, codebook [2^L, V].

    ``workspace`` (a uint8 CUDA tensor of at least tcq_encode_vec_workspace_bytes
    for one block; more lets more blocks run at once) and ``out`` (an Encoded of
    int32 start [n], int32 bits [n, W] and float32 cost [n]) are allocated when
    not given."""
    torch = _torch()
    if x.dim() != 2 or x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor [n_blocks, T]")
    n, T = x.shape
    if d is not None and (d.shape != x.shape or d.dtype != torch.float32 or not d.is_contiguous()):
        raise ValueError("d must be None or a contiguous float32 tensor shaped like x")
    if codebook is not MAD and codebook.numel() != (1 << L) * V:
        raise ValueError("codebook must hold 2^L rows of V entries")
    W = max(tcq_words_per_block(k, T), 1)
    if out is None:
        out = Encoded(torch.empty(n, dtype=torch.int32, device=x.device),
                      torch.empty((n, W), dtype=torch.int32, device=x.device),
                      torch.empty(n, dtype=torch.float32, device=x.device))
    elif (out.start_state.numel() < n or out.bits.numel() < n * W or out.path_cost.numel() < n):
        raise ValueError("encode_vec: out is smaller than the blocks need")
    if workspace is None:
        nbytes = max(tcq_encode_vec_workspace_bytes(L, k, V, T, n, cb_dtype_of(codebook)), 256)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    else:
        ws = workspace
    _check(tcq_encode_vec(_ptr(x), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), L, k, V, T, n,
                          _ptr(out.start_state), _ptr(out.bits), _ptr(out.path_cost),
                          ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream_handle(stream)),
           "tcq_encode_vec")
    return out


def decode_vec(bits, start_state, codebook, L: int, k: int, V: int, T: int, out=None, stream=None):
    """Values [n_blocks, T] of the vector trellis (into ``out`` when given)."""
    torch = _torch()
    n = start_state.shape[0]
    W = tcq_words_per_block(k, T)
    if bits.numel() < n * max(W, 0):
        raise ValueError("decode_vec: bits holds fewer than n_blocks * W words")
    if out is None:
        out = torch.empty((n, T), dtype=torch.float32, device=bits.device)
    elif out.numel() < n * T or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("decode_vec: out must be a contiguous float32 tensor of n_blocks * T")
    _check(tcq_decode_vec(_ptr(bits), _ptr(start_state), _ptr(codebook), cb_dtype_of(codebook), L,
                          k, V, T, n, _ptr(out), _stream_handle(stream)), "tcq_decode_vec")
    return out


# ---------------------------------------------------------------------------
# batched 16-bit products and 8-bit checkpoints
#
# A wait inside a product is bounded: one that gives up leaves the call's outputs
# unspecified and a flag that device_errors() returns (no call synchronises to look).
# ---------------------------------------------------------------------------
@dataclass
class Packed8:
    """An 8-bit checkpoint of a 16-bit tensor [n, cols]: ``codes`` (int8 [n, cols];
    for "e4m3" the bytes of the numbers), ``scales`` (uint8 [n, ceil(cols / 32)], the
    exponent + 127 of each group's power of two) and the format's name."""

    codes: "object"
    scales: "object"
    format: str = "int8"


# These calls can be shorter than their checks, so the checks are few and plain: torch
# sizes compare with tuples, addresses and streams go to ctypes as integers.
def _rows(t, what: str):
    """(TCQ_X_*, n, columns, row stride) of a 2-D 16-bit CUDA tensor with unit-stride rows
    (the stride of one row, or of none, does not matter)."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D CUDA tensor with unit-stride rows")
    (n, cols), (ld, step) = t.shape, t.stride()
    if step != 1 and cols > 1 and n:
        raise ValueError(f"{what} must be a 2-D CUDA tensor with unit-stride rows")
    dtype, torch = t.dtype, _torch()
    if dtype == torch.bfloat16:
        xt = TCQ_X_BF16
    elif dtype == torch.float16:
        xt = TCQ_X_F16
    else:
        raise TypeError(f"{what} must be float16 or bfloat16, got {dtype}")
    return xt, n, cols, ld if n > 1 and cols else max(cols, 1)


def _choice(table, name, what):
    try:
        return table[name]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {name!r}") from None


def _check_out(out, shape, dtype, device, what) -> int:
    """The row stride of an array that the caller gave."""
    if out.shape != shape or out.dtype != dtype:
        raise ValueError(f"{what} must be a {dtype} tensor {list(shape)}")
    (n, cols), (ld, step) = shape, out.stride()
    if n and step != 1 and cols > 1:
        raise ValueError(f"{what} must have unit-stride rows")
    if n > 1 and cols and ld < cols:
        raise ValueError(f"{what}: rows overlap")
    _check_device(out, device, what)
    return ld if n > 1 and cols else max(cols, 1)


def _check_apart(out, ldo, t, ldt, what):
    """Refuses a 16-bit ``out`` that shares elements with ``t``, which other rows or tiles
    of the call still read.  Columns of one buffer may interleave."""
    a, b, wide, width = out.data_ptr(), t.data_ptr(), out.shape[1], t.shape[1]
    if (out.numel() == 0 or t.numel() == 0 or b >= a + 2 * ((out.shape[0] - 1) * ldo + wide) or
            a >= b + 2 * ((t.shape[0] - 1) * ldt + width)):
        return
    if out.shape[0] > 1 and ldo == ldt and 2 * wide <= (b - a) % (2 * ldo) <= 2 * (ldo - width):
        return
    raise ValueError(f"out overlaps {what}")


def _check_device(t, device, what):
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")


def _check_packed(p, n, cols, device, what):
    fmt = _choice(Q8_FORMATS, p.format, "format")
    codes, scales = p.codes, p.scales
    groups = (cols + 31) // 32
    if (codes.shape != (n, cols) or codes.element_size() != 1 or not codes.is_contiguous() or
            scales.shape != (n, groups) or scales.dtype != _torch().uint8 or not scales.is_contiguous()):
        raise ValueError(f"{what} must hold contiguous 8-bit codes [{n}, {cols}] and uint8 scales [{n}, {groups}]")
    _check_device(codes, device, what)
    _check_device(scales, device, what)
    return fmt


def _check_matrix(bits, start_state, scale, codebook, L, k, T, rows, cols, device, what):
    if not (1 <= k <= TCQ_MAX_K and 1 <= T <= TCQ_MAX_T):
        raise TCQError(TCQ_ERR_UNSUPPORTED, what)
    nb = rows * (cols // T)
    if bits.numel() < nb * ((T * k + 31) // 32) or start_state.numel() < nb:
        raise ValueError(f"{what}: tensors too small for a {rows} x {cols} matrix of T={T} blocks")
    if (bits.element_size() != 4 or start_state.element_size() != 4 or not bits.is_contiguous() or
            not start_state.is_contiguous()):
        raise ValueError(f"{what}: bits and start_state are contiguous 32-bit words")
    _check_device(bits, device, "bits")
    _check_device(start_state, device, "start_state")
    if scale is not None:
        if scale.numel() < nb or scale.dtype != _torch().float32 or not scale.is_contiguous():
            raise ValueError(f"{what}: scale must hold a contiguous float32 value per block")
        _check_device(scale, device, "scale")
    if codebook is not MAD:
        if codebook.numel() < (1 << L) or not codebook.is_contiguous():
            raise ValueError(f"{what}: codebook must hold 2^L contiguous entries")
        _check_device(codebook, device, "codebook")


def _empty(like, shape, dtype, stream):
    """Memory of the stream that will write it: a given one may run before what the
    current stream still does to memory freed there, and after this call has returned."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if stream.device != like.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {like.device}")
    with _torch().cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _scratch(workspace, nbytes, like, what, stream):
    if workspace is None:
        return _empty(like, nbytes or 1, _torch().uint8, stream)
    if workspace.device != like.device or workspace.dtype != _torch().uint8 or not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace must be a contiguous uint8 tensor on x's device")
    return workspace


def _addr(t):
    return None if t is None or t is MAD else t.data_ptr()


def _launch(what, device, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current, on the given stream or on
    that device's current one."""
    torch = _torch()
    index = device.index
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        handle = stream.cuda_stream
    else:
        handle = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != TCQ_OK:
        raise TCQError(status, what)


@functools.lru_cache(maxsize=1024)
def _sized(device, query, *args) -> int:
    """A workspace query, a function of the shape and the device (whose multiprocessors it
    counts)."""
    with _torch().cuda.device(device):
        return getattr(load_library(), query)(*args)


def pack8(x, format: str = "int8", out: Packed8 | None = None, stream=None) -> Packed8:
    """8-bit checkpoint of ``x`` (float16 or bfloat16 CUDA [n, cols], unit-stride rows)."""
    torch, lib = _torch(), load_library()
    xt, n, cols, ld = _rows(x, "x")
    if out is None:
        fmt = _choice(Q8_FORMATS, format, "format")
        out = Packed8(_empty(x, (n, cols), torch.int8, stream),
                      _empty(x, (n, (cols + 31) // 32), torch.uint8, stream), format)
    else:
        fmt = _check_packed(out, n, cols, x.device, "out")
    _launch("tcq_pack8", x.device, stream, lib.tcq_pack8, x.data_ptr(), xt, ld, n, cols, fmt,
            out.codes.data_ptr(), out.scales.data_ptr())
    return out


def unpack8(packed: Packed8, dtype=None, out=None, stream=None):
    """The values of an 8-bit checkpoint, as ``dtype`` (bfloat16 when not given) [n, cols]."""
    torch, lib = _torch(), load_library()
    codes = packed.codes
    if codes.dim() != 2 or not codes.is_cuda:
        raise ValueError("packed must hold CUDA tensors [n, cols]")
    n, cols = codes.shape
    dev = codes.device
    fmt = _check_packed(packed, n, cols, dev, "packed")
    if out is None:
        out = _empty(codes, (n, cols), dtype or torch.bfloat16, stream)
    else:
        _check_out(out, (n, cols), dtype or out.dtype, dev, "out")
    xt, _, _, ld = _rows(out, "out")
    _launch("tcq_unpack8", dev, stream, lib.tcq_unpack8, codes.data_ptr(), packed.scales.data_ptr(), fmt, n, cols,
            out.data_ptr(), xt, ld)
    return out


def gemm(bits, start_state, scale, codebook, L: int, k: int, T: int, rows: int, cols: int, x, bias=None,
         act: str = "none", residual=None, checkpoint=None, out=None, workspace=None, stream=None):
    """act(x W^T + bias) + residual for a trellis-coded W [rows, cols] (gemv's blocks)
    and ``x`` float16 or bfloat16 [n, cols]; [n, rows] of x's type.

    ``bias`` float32 [rows]; ``residual`` like the result; ``checkpoint`` a Packed8 of
    [n, rows] that receives the pre-activation in 8 bits.  ``workspace`` (uint8, at
    least tcq_gemm_workspace_bytes) and ``out`` are allocated when not given; ``out`` may
    be ``residual`` itself, and overlaps neither ``x`` nor a part of ``residual``.

    Sums are fp32; how a weight (scale times codeword) enters them depends on the number of
    tokens, so that a token's result may differ in its last bits with the batch it comes in:
    fp32 for a single token without a checkpoint, rounded to binary16 (relative to powers of
    two of its row and the table) for 2 to 256 and for any number of float16 ones, rounded
    to bfloat16 for more than 256 bfloat16 tokens."""
    torch, lib = _torch(), load_library()
    xt, n, width, ldx = _rows(x, "x")
    dev, dtype = x.device, x.dtype
    if width != cols:
        raise ValueError(f"gemm: x has {width} columns, the matrix {cols}")
    a = _choice(ACTIVATIONS, act, "act")
    _check_matrix(bits, start_state, scale, codebook, L, k, T, rows, cols, dev, "gemm")
    if bias is not None:
        if bias.numel() != rows or bias.dtype != torch.float32 or not bias.is_contiguous():
            raise ValueError("gemm: bias must be a contiguous float32 tensor [rows]")
        _check_device(bias, dev, "bias")
    ldr = 0
    if residual is not None:
        ldr = _check_out(residual, (n, rows), dtype, dev, "residual")
    if out is None:
        out, ldy = _empty(x, (n, rows), dtype, stream), max(rows, 1)
    else:
        ldy = _check_out(out, (n, rows), dtype, dev, "out")
        _check_apart(out, ldy, x, ldx, "x")
        if residual is not None and (residual.data_ptr() != out.data_ptr() or ldr != ldy):
            _check_apart(out, ldy, residual, ldr, "a part of residual")
    zc = zs = None
    zf = TCQ_Q8_INT8
    if checkpoint is not None:
        zf = _check_packed(checkpoint, n, rows, dev, "checkpoint")
        zc, zs = checkpoint.codes.data_ptr(), checkpoint.scales.data_ptr()
    cb = cb_dtype_of(codebook)
    wp, wb = None, 0
    if n != 1 or zc is not None:
        ws = _scratch(workspace, _sized(dev, "tcq_gemm_workspace_bytes", L, k, T, rows, cols, n, cb), x, "gemm",
                      stream)
        wp, wb = ws.data_ptr(), ws.numel()
    _launch("tcq_gemm", dev, stream, lib.tcq_gemm, bits.data_ptr(), start_state.data_ptr(), _addr(scale),
            _addr(codebook), cb, L, k, T, rows, cols, x.data_ptr(), xt, ldx, n, _addr(bias), a, _addr(residual),
            ldr, out.data_ptr(), ldy, zc, zs, zf, wp, wb)
    return out


def gemm_dgrad(bits, start_state, scale, codebook, L: int, k: int, T: int, rows: int, cols: int, dz, out=None,
               workspace=None, stream=None):
    """dz W for a trellis-coded W [rows, cols] and ``dz`` float16 or bfloat16 [n, rows];
    [n, cols] of dz's type.  ``out`` must not overlap ``dz``.  Weights are rounded like
    ``gemm``'s, those of a single token to binary16."""
    lib = load_library()
    xt, n, width, lddz = _rows(dz, "dz")
    dev = dz.device
    if width != rows:
        raise ValueError(f"gemm_dgrad: dz has {width} columns, the matrix {rows} rows")
    _check_matrix(bits, start_state, scale, codebook, L, k, T, rows, cols, dev, "gemm_dgrad")
    if out is None:
        out, lddx = _empty(dz, (n, cols), dz.dtype, stream), max(cols, 1)
    else:
        lddx = _check_out(out, (n, cols), dz.dtype, dev, "out")
        _check_apart(out, lddx, dz, lddz, "dz")
    cb = cb_dtype_of(codebook)
    ws = _scratch(workspace, _sized(dev, "tcq_gemm_dgrad_workspace_bytes", L, k, T, rows, cols, n, cb), dz,
                  "gemm_dgrad", stream)
    _launch("tcq_gemm_dgrad", dev, stream, lib.tcq_gemm_dgrad, bits.data_ptr(), start_state.data_ptr(), _addr(scale),
            _addr(codebook), cb, L, k, T, rows, cols, dz.data_ptr(), xt, lddz, n, out.data_ptr(), lddx,
            ws.data_ptr(), ws.numel())
    return out


def act_grad8(dy, checkpoint, act: str, dbias: bool = True, out=None, workspace=None, stream=None):
    """(dz, dbias): dy act'(z) in dy's type [n, rows] and its float32 column sums (None
    unless ``dbias``), from the 8-bit checkpoint of the pre-activation (None for act
    "none").  ``out`` may be ``dy``."""
    torch, lib = _torch(), load_library()
    xt, n, rows, lddy = _rows(dy, "dy")
    dev = dy.device
    a = _choice(ACTIVATIONS, act, "act")
    zc = zs = None
    zf = TCQ_Q8_INT8
    if checkpoint is not None:
        zf = _check_packed(checkpoint, n, rows, dev, "checkpoint")
        zc, zs = checkpoint.codes.data_ptr(), checkpoint.scales.data_ptr()
    elif a != TCQ_ACT_NONE:
        raise ValueError(f"act_grad8: {act!r} needs the checkpoint of the pre-activation")
    if out is None:
        out, lddz = _empty(dy, (n, rows), dy.dtype, stream), max(rows, 1)
    else:
        lddz = _check_out(out, (n, rows), dy.dtype, dev, "out")
        if out.data_ptr() != dy.data_ptr() or lddz != lddy:
            _check_apart(out, lddz, dy, lddy, "a part of dy")
    db, dp, wp, wb = None, None, None, 0
    if dbias:
        db = _empty(dy, rows, torch.float32, stream)
        ws = _scratch(workspace, _sized(dev, "tcq_act_grad8_workspace_bytes", n, rows), dy, "act_grad8", stream)
        dp, wp, wb = db.data_ptr(), ws.data_ptr(), ws.numel()
    _launch("tcq_act_grad8", dev, stream, lib.tcq_act_grad8, dy.data_ptr(), xt, lddy, zc, zs, zf, a, n, rows,
            out.data_ptr(), lddz, dp, wp, wb)
    return out, db


def wgrad8(dz, packed: Packed8, out=None, accumulate: bool = False, workspace=None, stream=None):
    """dz^T x, float32 [rows, cols], for ``dz`` float16 or bfloat16 [n, rows] and the
    8-bit checkpoint of x [n, cols]; added to ``out`` when ``accumulate``."""
    torch, lib = _torch(), load_library()
    xt, n, rows, lddz = _rows(dz, "dz")
    dev = dz.device
    if packed.codes.dim() != 2:
        raise ValueError("packed must hold CUDA tensors [n, cols]")
    cols = packed.codes.shape[1]
    fmt = _check_packed(packed, n, cols, dev, "packed")
    if out is None:
        if accumulate:
            raise ValueError("wgrad8: accumulate needs out")
        out, lddw = _empty(dz, (rows, cols), torch.float32, stream), max(cols, 1)
    else:
        lddw = _check_out(out, (rows, cols), torch.float32, dev, "out")
    ws = _scratch(workspace, _sized(dev, "tcq_wgrad8_workspace_bytes", rows, cols, n), dz, "wgrad8", stream)
    _launch("tcq_wgrad8", dev, stream, lib.tcq_wgrad8, dz.data_ptr(), xt, lddz, packed.codes.data_ptr(),
            packed.scales.data_ptr(), fmt, n, rows, cols, out.data_ptr(), lddw, int(accumulate), ws.data_ptr(),
            ws.numel())
    return out


def ub8_encode(x, d, codebook, V: int, m: int, fixed_start=None, out=None,
               stream=None) -> Encoded:
    """TCQ over the 8-state set-partitioned trellis of every row of ``x`` (fp32
    CUDA [n_blocks, T], T / V steps of V weights); ``codebook`` holds 4 * 2^m rows
    of V values (row r in subset r mod 4).  A free start state per block, or the
    int32 tensor ``fixed_start``."""
    torch = _torch()
    if x.dim() != 2 or x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor [n_blocks, T]")
    n, T = x.shape
    if d is not None and (d.shape != x.shape or d.dtype != torch.float32 or not d.is_contiguous()):
        raise ValueError("d must be None or a contiguous float32 tensor shaped like x")
    if codebook is MAD or codebook.numel() != (4 << m) * V:
        raise ValueError("codebook must be a table of 4 * 2^m rows of V entries")
    W = tcq_ub8_words_per_block(V, m, T)
    if W < 0:
        raise TCQError(TCQ_ERR_UNSUPPORTED, "tcq_ub8_words_per_block")
    if out is None:
        out = Encoded(torch.empty(n, dtype=torch.int32, device=x.device),
                      torch.empty((n, W), dtype=torch.int32, device=x.device),
                      torch.empty(n, dtype=torch.float32, device=x.device))
    elif out.start_state.numel() < n or out.bits.numel() < n * W or out.path_cost.numel() < n:
        raise ValueError("ub8_encode: out is smaller than the blocks need")
    if fixed_start is not None and (fixed_start.numel() < n or fixed_start.dtype != torch.int32
                                    or not fixed_start.is_cuda):
        raise ValueError("fixed_start must be an int32 CUDA tensor of n_blocks start states")
    _check(tcq_ub8_encode(_ptr(x), _ptr(d), _ptr(codebook), cb_dtype_of(codebook), V, m, T, n,
                          _ptr(fixed_start), _ptr(out.start_state), _ptr(out.bits),
                          _ptr(out.path_cost), _stream_handle(stream)), "tcq_ub8_encode")
    return out


def ub8_decode(bits, start_state, codebook, V: int, m: int, T: int, out=None, stream=None):
    """Values [n_blocks, T] of 8-state set-partitioned trellis streams."""
    torch = _torch()
    n = start_state.shape[0]
    W = tcq_ub8_words_per_block(V, m, T)
    if W < 0:
        raise TCQError(TCQ_ERR_UNSUPPORTED, "tcq_ub8_words_per_block")
    if bits.numel() < n * W:
        raise ValueError("ub8_decode: bits holds fewer than n_blocks * W words")
    if codebook is MAD or codebook.numel() != (4 << m) * V:
        raise ValueError("codebook must be a table of 4 * 2^m rows of V entries")
    if out is None:
        out = torch.empty((n, T), dtype=torch.float32, device=bits.device)
    elif out.numel() < n * T or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("ub8_decode: out must be a contiguous float32 tensor of n_blocks * T")
    _check(tcq_ub8_decode(_ptr(bits), _ptr(start_state), _ptr(codebook), cb_dtype_of(codebook), V,
                          m, T, n, _ptr(out), _stream_handle(stream)), "tcq_ub8_decode")
    return out


def host_pipeline_parts(n_blocks: int, chunks: int, sm_count: int):
    """Block ranges [lo, hi) of HostPipeline: a short lead part (1 / (8 chunks)
    of the blocks) and ``chunks`` equal parts, one part when ``chunks`` is 1.
    For large inputs the sizes are whole waves of the encoder (8 blocks per SM:
    every grouped configuration runs 1, 2, 4 or 8 blocks per SM at a time), so
    that only the last part ends on a partly filled round."""
    chunks = max(1, chunks)
    wave = 8 * max(1, sm_count)
    lead = min(n_blocks, -(-n_blocks // (8 * chunks))) if chunks > 1 else 0
    per = max(1, -(-(n_blocks - lead) // chunks))
    if n_blocks >= 8 * chunks * wave:
        lead = -(-lead // wave) * wave
        per = -(-per // wave) * wave
    return ([(0, lead)] if lead else []) + [(lo, min(n_blocks, lo + per)) for lo in range(lead, n_blocks, per)]


class HostPipeline:
    """End-to-end encode of host arrays: pinned host -> device -> encode -> host.

    Buffers are allocated once.  ``run`` splits the blocks into a short lead
    part (1 / (8 chunks) of them) and ``chunks`` equal parts (one part when
    ``chunks`` is 1): a copy stream
    brings part i + 1's inputs in while the compute stream encodes and decodes
    part i, and takes part i's start states, bits and costs back while part i + 1
    is encoded, so only the lead part's input copy (short, so that the encoder
    starts early; the next part's copy hides behind its encode) and the last
    part's output copy are not hidden behind the encoder.
    """

    def __init__(self, n_blocks: int, T: int, L: int, k: int, weighted: bool, codebook_host,
                 device=None, with_decode: bool = True, chunks: int = 8):
        torch = _torch()
        dev = torch.device(device or "cuda")
        self.L, self.k, self.T, self.n = L, k, T, n_blocks
        W = tcq_words_per_block(k, T)
        self.x_dev = torch.empty((n_blocks, T), dtype=torch.float32, device=dev)
        self.d_dev = torch.empty((n_blocks, T), dtype=torch.float32, device=dev) if weighted else None
        self.cb_dev = codebook_host.to(dev)
        self.parts = host_pipeline_parts(n_blocks, chunks,
                                         torch.cuda.get_device_properties(dev).multi_processor_count)
        self.ws = Workspace(L, k, T, max(hi - lo for lo, hi in self.parts), cb_dtype_of(self.cb_dev), dev)
        self.enc = Encoded(torch.empty(n_blocks, dtype=torch.int32, device=dev),
                           torch.empty((n_blocks, W), dtype=torch.int32, device=dev),
                           torch.empty(n_blocks, dtype=torch.float32, device=dev))
        self.y_dev = torch.empty((n_blocks, T), dtype=torch.float32, device=dev) if with_decode else None
        self.start_h = torch.empty(n_blocks, dtype=torch.int32, pin_memory=True)
        self.bits_h = torch.empty((n_blocks, W), dtype=torch.int32, pin_memory=True)
        self.cost_h = torch.empty(n_blocks, dtype=torch.float32, pin_memory=True)
        self.copy_stream = torch.cuda.Stream(device=dev)
        self.ev_in = [torch.cuda.Event() for _ in self.parts]
        self.ev_done = [torch.cuda.Event() for _ in self.parts]

    def h2d_bytes(self) -> int:
        return self.x_dev.numel() * 4 + (self.d_dev.numel() * 4 if self.d_dev is not None else 0)

    def d2h_bytes(self) -> int:
        return (self.start_h.numel() + self.bits_h.numel() + self.cost_h.numel()) * 4

    def run(self, x_pinned, d_pinned=None, stream=None):
        torch = _torch()
        cs = self.copy_stream
        ms = stream or torch.cuda.current_stream()
        cs.wait_stream(ms)  # the previous run's readers of these buffers are done

        def copy_in(i):
            lo, hi = self.parts[i]
            with torch.cuda.stream(cs):
                self.x_dev[lo:hi].copy_(x_pinned[lo:hi], non_blocking=True)
                if self.d_dev is not None:
                    self.d_dev[lo:hi].copy_(d_pinned[lo:hi], non_blocking=True)
                self.ev_in[i].record(cs)

        copy_in(0)
        for i, (lo, hi) in enumerate(self.parts):
            if i + 1 < len(self.parts):
                copy_in(i + 1)
            ms.wait_event(self.ev_in[i])
            part = Encoded(self.enc.start_state[lo:hi], self.enc.bits[lo:hi], self.enc.path_cost[lo:hi])
            encode(self.x_dev[lo:hi], None if self.d_dev is None else self.d_dev[lo:hi], self.cb_dev,
                   self.L, self.k, self.ws, part, ms)
            if self.y_dev is not None:
                decode(part.bits, part.start_state, self.cb_dev, self.L, self.k, self.T,
                       self.y_dev[lo:hi], ms)
            self.ev_done[i].record(ms)
            with torch.cuda.stream(cs):
                cs.wait_event(self.ev_done[i])
                self.start_h[lo:hi].copy_(part.start_state, non_blocking=True)
                self.bits_h[lo:hi].copy_(part.bits, non_blocking=True)
                self.cost_h[lo:hi].copy_(part.path_cost, non_blocking=True)
        ms.wait_stream(cs)
        return self.start_h, self.bits_h, self.cost_h


def tcq_encode_static_scratch(x, d, codebook, cb_dtype, L, k, T, n_blocks, start_state, bits,
                              path_cost, stream) -> int:
    """The allocation-free encoder (scratch in a static device array of the library)."""
    fn = _static_scratch_fn()
    return int(fn(x, d, codebook, cb_dtype, L, k, T, n_blocks, start_state, bits, path_cost,
                  stream))


def _static_scratch_fn():
    lib = load_library()
    fn = lib.tcq_encode_static_scratch
    if fn.argtypes is None:
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        fn.argtypes = [vp, vp, vp, ci, ci, ci, ci, i64, vp, vp, vp, vp]
        fn.restype = ci
    return fn
