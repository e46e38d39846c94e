"""ctypes binding of libgptq_mi355x.so (the C ABI in include/gptq.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch provides device memory and streams. If the library is not
built, importing this module raises ImportError: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq_mi355x.so")

GPTQ_OK = 0
GPTQ_ERR_INVALID_ARG = 1
GPTQ_ERR_WORKSPACE = 2
GPTQ_ERR_NOT_PD = 3
GPTQ_ERR_HIP = 4
GPTQ_ERR_UNSUPPORTED = 5

GPTQ_DTYPE_F16 = 0
GPTQ_DTYPE_F32 = 1

OP_ACCUMULATE = 0
OP_PREPARE = 1
OP_QUANTIZE = 2
OP_QUANTIZE_PERM = 3
OP_FORWARD_ADAPTERS = 4
OP_BACKWARD = 5
OP_HEAD_LOSS = 6
OP_HEAD_BACKWARD = 7

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950) first")

# PyTorch-ROCm ships its own libamdhip64.so.7. Importing torch first makes the
# dynamic loader bind the library's libamdhip64.so.7 dependency to that
# already-loaded runtime, so torch's streams and allocations and the
# library's launches live in one HIP runtime.
import torch  # noqa: E402,F401

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_sz = ctypes.c_size_t

lib.gptq_version.restype = _int
lib.gptq_version.argtypes = []
lib.gptq_status_string.restype = ctypes.c_char_p
lib.gptq_status_string.argtypes = [_int]
lib.gptq_workspace_bytes.restype = _sz
lib.gptq_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
lib.gptq_hessian_accumulate.restype = _int
lib.gptq_hessian_accumulate.argtypes = [_p, _i64, _p, _i64, _i64, ctypes.c_float, _p, _sz, _p]
lib.gptq_prepare_hinv.restype = _int
lib.gptq_prepare_hinv.argtypes = [_p, _i64, ctypes.c_double, _p, _p, _sz,
                                  ctypes.POINTER(ctypes.c_int64), _p]
lib.gptq_quantize_layer.restype = _int
lib.gptq_quantize_layer.argtypes = [_p, _int, _i64, _i64, _i64, _p, _int, _int, _int,
                                    _p, _p, _p, _p, _p, _sz, _p]
lib.gptq_act_order.restype = _int
lib.gptq_act_order.argtypes = [_p, _i64, _p, _p]
lib.gptq_prepare_hinv_three_step.restype = _int
lib.gptq_prepare_hinv_three_step.argtypes = lib.gptq_prepare_hinv.argtypes
lib.gptq_prepare_hinv_perm.restype = _int
lib.gptq_prepare_hinv_perm.argtypes = [_p, _i64, _p, ctypes.c_double, _p, _p, _sz,
                                       ctypes.POINTER(ctypes.c_int64), _p]
lib.gptq_packed_words.restype = _i64
lib.gptq_packed_words.argtypes = [_i64, _int]
lib.gptq_pack_codes.restype = _int
lib.gptq_pack_codes.argtypes = [_p, _i64, _i64, _int, _p, _p]
lib.gptq_dequant_gemm.restype = _int
lib.gptq_dequant_gemm.argtypes = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int, _p, _p,
                                  _i64, _p]
lib.gptq_linear_forward.restype = _int
lib.gptq_linear_forward.argtypes = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int, _int, _p,
                                    _i64, _p]
lib.gptq_hessian_accumulate_noalloc.restype = _int
lib.gptq_hessian_accumulate_noalloc.argtypes = [_p, _i64, _p, _i64, _i64, ctypes.c_float, _p]
lib.gptq_quantize_layer_perm.restype = _int
lib.gptq_quantize_layer_perm.argtypes = [_p, _int, _i64, _i64, _i64, _p, _p, _int, _int, _int,
                                         _p, _p, _p, _p, _p, _p, _sz, _p]


class _Adapters(ctypes.Structure):  # gptq_adapters
    _fields_ = [("A", _p), ("B", _p), ("scaling", _p), ("index", _p), ("count", _i64),
                ("rank", _int)]


_f = ctypes.c_float
_ad = ctypes.POINTER(_Adapters)
lib.gptq_adapters_workspace_bytes.restype = _sz
lib.gptq_adapters_workspace_bytes.argtypes = [_int, _i64, _i64, _i64, _i64, _int]
lib.gptq_head_workspace_bytes.restype = _sz
lib.gptq_head_workspace_bytes.argtypes = [_int, _i64, _i64, _i64, _int]
lib.gptq_dequant_gemm_adapters.restype = _int
lib.gptq_dequant_gemm_adapters.argtypes = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int, _p,
                                           _ad, _p, _i64, _p, _sz, _p]
lib.gptq_linear_forward_adapters.restype = _int
lib.gptq_linear_forward_adapters.argtypes = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int,
                                             _int, _ad, _p, _i64, _p, _sz, _p]
lib.gptq_linear_backward.restype = _int
lib.gptq_linear_backward.argtypes = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int, _p, _ad,
                                     _p, _i64, _p, _i64, _p, _p, _p, _sz, _p]
_head = [_p, _i64, _i64, _i64, _p, _int, _i64, _p, _p, _int]  # h and the layer
lib.gptq_head_loss.restype = _int
lib.gptq_head_loss.argtypes = _head + [_p, _p, _p, _p, _p, _sz, _p]
lib.gptq_head_loss_backward.restype = _int
lib.gptq_head_loss_backward.argtypes = _head + [_p, _p, _p, _p, _p, _i64, _p, _sz, _p]
lib.gptq_head_distill.restype = _int
lib.gptq_head_distill.argtypes = _head + [_p, _p, _int, _f, _p, _p, _p, _p, _sz, _p]
lib.gptq_head_distill_backward.restype = _int
lib.gptq_head_distill_backward.argtypes = _head + [_p, _p, _int, _f, _p, _p, _p, _p, _i64, _p, _sz,
                                                   _p]


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str, info: int = 0):
        name = lib.gptq_status_string(status).decode()
        msg = f"{where}: {name}"
        if info:
            msg += f" (info={info})"
        super().__init__(msg)
        self.status = status
        self.info = info


def status_string(status: int) -> str:
    return lib.gptq_status_string(status).decode()


def version() -> int:
    return lib.gptq_version()


def workspace_bytes(op: int, rows: int, cols: int, n: int) -> int:
    return int(lib.gptq_workspace_bytes(op, rows, cols, n))


# ---------------------------------------------------------------- torch layer
def _torch():
    import torch
    return torch


def _stream_ptr(stream, device) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _workspace(nbytes: int, device, workspace=None, stream=None):
    """The caller's workspace (checked), or a temporary one. A temporary is
    freed when the call returns while its kernels may still run; torch's
    caching allocator keeps it from being reused before the work queued on
    the current stream ends, and record_stream extends that to `stream`."""
    torch = _torch()
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        if workspace.device != device or workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small or on another device")
        if workspace.data_ptr() % 256:
            raise ValueError("workspace must be 256-byte aligned")
        return workspace, workspace.numel() * workspace.element_size()
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    if stream is not None and stream != torch.cuda.current_stream(device):
        ws.record_stream(stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    return ws, nbytes


def _check_out(t, shape, dtype, device, name):
    """A preallocated output must match exactly: the library writes
    prod(shape) elements of dtype from its data pointer."""
    if t is None or t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}")
    return t


def _check(status: int, where: str, info: int = 0):
    if status != GPTQ_OK:
        raise GPTQError(status, where, info)


def hessian_accumulate(H, X, alpha: float = 2.0, workspace=None, stream=None):
    """H += alpha * X^T X on the GPU. H: d x d fp32 (contiguous), X: n x d fp16
    with unit column stride. Returns H."""
    torch = _torch()
    if H.dtype != torch.float32 or not H.is_cuda or not H.is_contiguous():
        raise ValueError("H must be a contiguous fp32 CUDA tensor")
    if X.dtype != torch.float16 or X.device != H.device or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D fp16 CUDA tensor with unit column stride")
    d = H.shape[0]
    if H.shape != (d, d) or X.shape[1] != d:
        raise ValueError("shape mismatch")
    n = X.shape[0]
    ldx = X.stride(0) if n > 1 else d
    ws, wsb = _workspace(workspace_bytes(OP_ACCUMULATE, 0, d, n), H.device, workspace, stream)
    st = lib.gptq_hessian_accumulate(H.data_ptr(), d, X.data_ptr(), n, ldx, alpha,
                                     ws.data_ptr() if ws is not None else None, wsb,
                                     _stream_ptr(stream, H.device))
    _check(st, "gptq_hessian_accumulate")
    return H


def hessian_accumulate_noalloc(H, X, alpha: float = 2.0, stream=None):
    """H += alpha * X^T X like hessian_accumulate, with no workspace and no
    allocation (gptq_hessian_accumulate_noalloc). Returns H."""
    torch = _torch()
    if H.dtype != torch.float32 or not H.is_cuda or not H.is_contiguous():
        raise ValueError("H must be a contiguous fp32 CUDA tensor")
    if X.dtype != torch.float16 or X.device != H.device or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D fp16 CUDA tensor with unit column stride")
    d = H.shape[0]
    if H.shape != (d, d) or X.shape[1] != d:
        raise ValueError("shape mismatch")
    n = X.shape[0]
    ldx = X.stride(0) if n > 1 else d
    st = lib.gptq_hessian_accumulate_noalloc(H.data_ptr(), d, X.data_ptr(), n, ldx, alpha,
                                             _stream_ptr(stream, H.device))
    _check(st, "gptq_hessian_accumulate_noalloc")
    return H


def _check_H(H):
    torch = _torch()
    if H.dtype != torch.float32 or not H.is_cuda or not H.is_contiguous() or H.dim() != 2:
        raise ValueError("H must be a contiguous fp32 CUDA tensor")
    if H.shape[0] != H.shape[1]:
        raise ValueError("H must be square")
    return H.shape[0]


def _check_perm(perm, n, device):
    torch = _torch()
    if perm is None:
        return None
    if perm.dtype != torch.int32 or perm.device != device or perm.shape != (n,) or \
            not perm.is_contiguous():
        raise ValueError(f"perm must be a contiguous int32 tensor of length {n} on {device}")
    return perm


def prepare_hinv(H, percdamp: float = 0.01, out=None, workspace=None, stream=None):
    """Hinv (d x d fp32, upper triangular) from H. Raises GPTQError with
    status GPTQ_ERR_NOT_PD and the failing pivot in .info."""
    return prepare_hinv_perm(H, None, percdamp, out, workspace, stream)


def prepare_hinv_three_step(H, percdamp: float = 0.01, out=None, workspace=None, stream=None):
    """prepare_hinv through the pages' three steps (Cholesky, inverse through
    the factor, upper Cholesky of the inverse): gptq_prepare_hinv_three_step."""
    torch = _torch()
    d = _check_H(H)
    if out is None:
        out = torch.empty((d, d), dtype=torch.float32, device=H.device)
    _check_out(out, (d, d), torch.float32, H.device, "out")
    ws, wsb = _workspace(workspace_bytes(OP_PREPARE, 0, d, 0), H.device, workspace, stream)
    info = ctypes.c_int64(0)
    st = lib.gptq_prepare_hinv_three_step(H.data_ptr(), d, float(percdamp), out.data_ptr(),
                                          ws.data_ptr(), wsb, ctypes.byref(info),
                                          _stream_ptr(stream, H.device))
    _check(st, "gptq_prepare_hinv_three_step", info.value)
    return out


def act_order(H, out=None, stream=None):
    """perm (d int32): the columns in decreasing order of H's diagonal, ties
    by index (gptq_act_order)."""
    torch = _torch()
    d = _check_H(H)
    if out is None:
        out = torch.empty((d,), dtype=torch.int32, device=H.device)
    _check_perm(out, d, H.device)
    st = lib.gptq_act_order(H.data_ptr(), d, out.data_ptr(), _stream_ptr(stream, H.device))
    _check(st, "gptq_act_order")
    return out


def prepare_hinv_perm(H, perm, percdamp: float = 0.01, out=None, workspace=None, stream=None):
    """Hinv of H with rows and columns taken in the order perm (None: the
    identity, i.e. gptq_prepare_hinv). H must hold both triangles."""
    torch = _torch()
    d = _check_H(H)
    perm = _check_perm(perm, d, H.device)
    if out is None:
        out = torch.empty((d, d), dtype=torch.float32, device=H.device)
    _check_out(out, (d, d), torch.float32, H.device, "out")
    ws, wsb = _workspace(workspace_bytes(OP_PREPARE, 0, d, 0), H.device, workspace, stream)
    info = ctypes.c_int64(0)
    st_ptr = _stream_ptr(stream, H.device)
    if perm is None:
        st = lib.gptq_prepare_hinv(H.data_ptr(), d, float(percdamp), out.data_ptr(),
                                   ws.data_ptr(), wsb, ctypes.byref(info), st_ptr)
        _check(st, "gptq_prepare_hinv", info.value)
    else:
        st = lib.gptq_prepare_hinv_perm(H.data_ptr(), d, perm.data_ptr(), float(percdamp),
                                        out.data_ptr(), ws.data_ptr(), wsb, ctypes.byref(info),
                                        st_ptr)
        _check(st, "gptq_prepare_hinv_perm", info.value)
    return out


def quantize_layer(W, Hinv, bits: int = 4, groupsize: int = 128, blocksize: int = 128,
                   out=None, workspace=None, stream=None):
    """GPTQ sweep. W: rows x cols fp16/fp32 (unit column stride); Hinv from
    prepare_hinv; groupsize <= 0 means one group per row (per-channel).
    Returns (codes uint8, scales fp32, zeros fp32, losses fp32)."""
    torch = _torch()
    if W.dim() != 2 or W.stride(1) != 1 or not W.is_cuda:
        raise ValueError("W must be a 2-D CUDA tensor with unit column stride")
    if W.dtype == torch.float16:
        wdt = GPTQ_DTYPE_F16
    elif W.dtype == torch.float32:
        wdt = GPTQ_DTYPE_F32
    else:
        raise ValueError("W must be fp16 or fp32")
    rows, cols = W.shape
    if Hinv.shape != (cols, cols) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous cols x cols fp32 tensor")
    if groupsize <= 0:  # per-channel: one group over all columns
        groupsize = cols
    g = groupsize
    ng = (cols + g - 1) // g
    dev = W.device
    if out is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, ng), dtype=torch.float32, device=dev)
        zeros = torch.empty((rows, ng), dtype=torch.float32, device=dev)
        losses = torch.empty((cols,), dtype=torch.float32, device=dev)
    else:
        codes, scales, zeros, losses = out
    _check_out(codes, (rows, cols), torch.uint8, dev, "codes")
    _check_out(scales, (rows, ng), torch.float32, dev, "scales")
    _check_out(zeros, (rows, ng), torch.float32, dev, "zeros")
    _check_out(losses, (cols,), torch.float32, dev, "losses")
    ws, wsb = _workspace(workspace_bytes(OP_QUANTIZE, rows, cols, 0), dev, workspace, stream)
    ldw = W.stride(0) if rows > 1 else cols
    st = lib.gptq_quantize_layer(W.data_ptr(), wdt, rows, cols, ldw, Hinv.data_ptr(), bits,
                                 groupsize, blocksize, codes.data_ptr(), scales.data_ptr(),
                                 zeros.data_ptr(), losses.data_ptr(), ws.data_ptr(), wsb,
                                 _stream_ptr(stream, dev))
    _check(st, "gptq_quantize_layer")
    return codes, scales, zeros, losses


def quantize_layer_perm(W, perm, Hinv, bits: int = 4, groupsize: int = 128, blocksize: int = 128,
                        out=None, workspace=None, stream=None):
    """Act-order sweep: W's columns processed in the order perm, with Hinv
    from prepare_hinv_perm(H, perm). Returns (codes, scales, zeros, losses,
    g_idx): codes, losses and g_idx (int32) in W's column order, scales and
    zeros per processing-order group."""
    torch = _torch()
    if W.dim() != 2 or W.stride(1) != 1 or not W.is_cuda:
        raise ValueError("W must be a 2-D CUDA tensor with unit column stride")
    if W.dtype == torch.float16:
        wdt = GPTQ_DTYPE_F16
    elif W.dtype == torch.float32:
        wdt = GPTQ_DTYPE_F32
    else:
        raise ValueError("W must be fp16 or fp32")
    rows, cols = W.shape
    perm = _check_perm(perm, cols, W.device)
    if Hinv.shape != (cols, cols) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous cols x cols fp32 tensor")
    if groupsize <= 0:  # per-channel: one group over all columns
        groupsize = cols
    g = groupsize
    ng = (cols + g - 1) // g
    dev = W.device
    if out is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, ng), dtype=torch.float32, device=dev)
        zeros = torch.empty((rows, ng), dtype=torch.float32, device=dev)
        losses = torch.empty((cols,), dtype=torch.float32, device=dev)
        g_idx = torch.empty((cols,), dtype=torch.int32, device=dev)
    else:
        codes, scales, zeros, losses, g_idx = out
    _check_out(codes, (rows, cols), torch.uint8, dev, "codes")
    _check_out(scales, (rows, ng), torch.float32, dev, "scales")
    _check_out(zeros, (rows, ng), torch.float32, dev, "zeros")
    _check_out(losses, (cols,), torch.float32, dev, "losses")
    if g_idx is not None:
        _check_out(g_idx, (cols,), torch.int32, dev, "g_idx")
    ws, wsb = _workspace(workspace_bytes(OP_QUANTIZE_PERM, rows, cols, 0), dev, workspace,
                         stream)
    ldw = W.stride(0) if rows > 1 else cols
    st = lib.gptq_quantize_layer_perm(W.data_ptr(), wdt, rows, cols, ldw,
                                      perm.data_ptr() if perm is not None else None,
                                      Hinv.data_ptr(), bits, groupsize, blocksize,
                                      codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                      losses.data_ptr(),
                                      g_idx.data_ptr() if g_idx is not None else None,
                                      ws.data_ptr(), wsb, _stream_ptr(stream, dev))
    _check(st, "gptq_quantize_layer_perm")
    return codes, scales, zeros, losses, g_idx


def packed_words(cols: int, bits: int) -> int:
    return int(lib.gptq_packed_words(cols, bits))


def pack_codes(codes, bits: int, out=None, stream=None):
    """rows x packed_words(cols, bits) int32 tensor holding the codes'
    uint32 words (gptq_pack_codes)."""
    torch = _torch()
    if codes.dtype != torch.uint8 or not codes.is_cuda or not codes.is_contiguous() or \
            codes.dim() != 2:
        raise ValueError("codes must be a contiguous 2-D uint8 CUDA tensor")
    rows, cols = codes.shape
    nw = packed_words(cols, bits)
    if out is None:
        out = torch.empty((rows, nw), dtype=torch.int32, device=codes.device)
    _check_out(out, (rows, nw), torch.int32, codes.device, "out")
    st = lib.gptq_pack_codes(codes.data_ptr(), rows, cols, bits, out.data_ptr(),
                             _stream_ptr(stream, codes.device))
    _check(st, "gptq_pack_codes")
    return out


def dequant_gemm(x, packed, bits: int, cols: int, scales, zeros, groupsize: int, g_idx=None,
                 out=None, stream=None):
    """y = x W_hat^T (m x rows fp32) for fp16 x (m x cols) and the packed
    codes with their scales and zeros (gptq_dequant_gemm)."""
    torch = _torch()
    if x.dtype != torch.float16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1 or \
            x.shape[1] != cols:
        raise ValueError("x must be an m x cols fp16 CUDA tensor with unit column stride")
    rows = packed.shape[0]
    if packed.dtype != torch.int32 or not packed.is_contiguous() or \
            packed.shape[1] != packed_words(cols, bits):
        raise ValueError("packed must come from pack_codes for these cols and bits")
    if groupsize <= 0:
        groupsize = cols
    ng = (cols + groupsize - 1) // groupsize
    for t in (scales, zeros):
        if t.dtype != torch.float32 or t.shape != (rows, ng) or not t.is_contiguous():
            raise ValueError("scales and zeros must be contiguous rows x ngroups fp32")
    g_idx = _check_perm(g_idx, cols, x.device)
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, rows), dtype=torch.float32, device=x.device)
    if out.dtype != torch.float32 or tuple(out.shape) != (m, rows) or out.device != x.device \
            or (m > 0 and out.stride(1) != 1):
        raise ValueError(f"out must be an {m} x {rows} fp32 tensor with unit column stride "
                         f"on {x.device}")
    ldx = x.stride(0) if m > 1 else cols
    st = lib.gptq_dequant_gemm(x.data_ptr(), m, cols, ldx, packed.data_ptr(), bits, rows,
                               scales.data_ptr(), zeros.data_ptr(), groupsize,
                               g_idx.data_ptr() if g_idx is not None else None, out.data_ptr(),
                               out.stride(0) if m > 1 else rows, _stream_ptr(stream, x.device))
    _check(st, "gptq_dequant_gemm")
    return out


def linear_forward(x, packed, bits: int, cols: int, scales, zeros, groupsize: int,
                   relu: bool = False, out=None, stream=None):
    """y = x W_hat^T, or max(x W_hat^T, 0) with relu, as m x rows fp16, for
    fp16 x (m x cols) and the 4- or 8-bit packed codes with their scales and
    zeros (gptq_linear_forward: the product for many tokens on MFMA)."""
    torch = _torch()
    if x.dtype != torch.float16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1 or \
            x.shape[1] != cols:
        raise ValueError("x must be an m x cols fp16 CUDA tensor with unit column stride")
    rows = packed.shape[0]
    if packed.dtype != torch.int32 or not packed.is_contiguous() or \
            packed.shape[1] != packed_words(cols, bits):
        raise ValueError("packed must come from pack_codes for these cols and bits")
    if groupsize <= 0:
        groupsize = cols
    ng = (cols + groupsize - 1) // groupsize
    for t in (scales, zeros):
        if t.dtype != torch.float32 or t.shape != (rows, ng) or not t.is_contiguous():
            raise ValueError("scales and zeros must be contiguous rows x ngroups fp32")
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, rows), dtype=torch.float16, device=x.device)
    elif out.dtype != torch.float16 or out.shape != (m, rows) or out.stride(1) != 1 or \
            out.device != x.device:
        raise ValueError("out must be an m x rows fp16 tensor with unit column stride")
    ldx = x.stride(0) if m > 1 else cols
    st = lib.gptq_linear_forward(x.data_ptr(), m, cols, ldx, packed.data_ptr(), bits, rows,
                                 scales.data_ptr(), zeros.data_ptr(), groupsize, 1 if relu else 0,
                                 out.data_ptr(), out.stride(0) if m > 1 else rows,
                                 _stream_ptr(stream, x.device))
    _check(st, "gptq_linear_forward")
    return out


# ------------------------------------------- adapters, gradients, vocabulary losses
# These calls are short enough on the GPU (a decode step of one token: 9 us)
# for their checks to count: tensors are compared by dtype identity, shape and
# device index, and workspace sizes, which depend on the sizes alone, are kept.
_f16, _f32, _i32 = torch.float16, torch.float32, torch.int32
# the current stream's handle without a Stream object (2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


@functools.lru_cache(maxsize=1024)
def adapters_workspace_bytes(op: int, m: int, rows: int, cols: int, count: int = 0,
                             rank: int = 0) -> int:
    """Workspace of OP_FORWARD_ADAPTERS or OP_BACKWARD for m tokens."""
    return int(lib.gptq_adapters_workspace_bytes(op, m, rows, cols, count, rank))


@functools.lru_cache(maxsize=1024)
def head_workspace_bytes(op: int, m: int, rows: int, cols: int, top: int = 1) -> int:
    """Workspace of OP_HEAD_LOSS or OP_HEAD_BACKWARD for m tokens and top
    entries each (labels: 1)."""
    return int(lib.gptq_head_workspace_bytes(op, m, rows, cols, top))


def _rows_of(t, m, n, dtype, dev, name):
    """An m x n matrix with unit column stride on GPU dev; returns its row stride."""
    if t.dtype is dtype and t.shape == (m, n) and t.get_device() == dev:
        ld, one = t.stride()
        if one == 1 or n <= 1 or m == 0:
            return ld if m > 1 else n
    raise ValueError(f"{name} must be an {m} x {n} {dtype} tensor with unit column stride "
                     f"on cuda:{dev}")


def _exactly(t, shape, dtype, dev, name):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} "
                         f"on cuda:{dev}")


def _input(x, n, name):
    """(tokens, row stride, GPU index) of an fp16 input with n columns (None: any)."""
    shape, dev = x.shape, x.get_device()
    if len(shape) == 2 and dev >= 0 and (n is None or shape[1] == n):
        return shape[0], _rows_of(x, *shape, _f16, dev, name), dev
    raise ValueError(f"{name} must be a 2-D fp16 CUDA tensor with unit column stride"
                     + ("" if n is None else f" and {n} columns"))


def _layer(packed, bits, cols, scales, zeros, groupsize, dev, g_idx=None):
    """The stored layer's checks; returns (rows, groupsize)."""
    if packed.dtype is not _i32 or packed.dim() != 2 or not packed.is_contiguous() or \
            packed.get_device() != dev or not 2 <= bits <= 8 or \
            packed.shape[1] != -(-cols // (32 // bits)):
        raise ValueError("packed must come from pack_codes for these cols and bits")
    rows = packed.shape[0]
    if groupsize <= 0:
        groupsize = cols
    shape = (rows, -(-cols // groupsize))
    _exactly(scales, shape, _f32, dev, "scales")
    _exactly(zeros, shape, _f32, dev, "zeros")
    if g_idx is not None:
        _exactly(g_idx, (cols,), _i32, dev, "g_idx")
    return rows, groupsize


def _adapters(A, B, scaling, index, m, rows, cols, dev):
    """The adapters' checks; returns the C struct."""
    if A.dim() != 3:
        raise ValueError("A must be count x rank x cols and B count x rows x rank")
    count, rank = A.shape[0], A.shape[1]
    _exactly(A, (count, rank, cols), _f16, dev, "A")
    _exactly(B, (count, rows, rank), _f16, dev, "B")
    _exactly(scaling, (count,), _f32, dev, "scaling")
    _exactly(index, (m,), _i32, dev, "index")
    return _Adapters(A.data_ptr(), B.data_ptr(), scaling.data_ptr(), index.data_ptr(), count, rank)


def _new(shape, dtype, dev, stream, result=True):
    """Memory for work on `stream`, from that stream's own pool: the current
    stream's may hand out blocks that its own queued work still uses. For a
    result the caller's stream is recorded, since it is read and freed there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if result:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _out_rows(out, m, n, dtype, dev, stream):
    """(out, its row stride), allocated when None."""
    if out is None:
        return _new((m, n), dtype, dev, stream), n
    return out, _rows_of(out, m, n, dtype, dev, "out")


def _out_exactly(out, shape, dtype, dev, name, stream):
    if out is None:
        return _new(shape, dtype, dev, stream)
    _exactly(out, shape, dtype, dev, name)
    return out


def _launch(fn, args, nbytes, dev, workspace, stream):
    """fn(*args, workspace, bytes, stream) on GPU dev; raises its errors."""
    ws = None
    if nbytes > 0:
        if workspace is None:
            # freed on return, for the next work on the same stream
            ws = _new(nbytes, torch.uint8, dev, stream, False)
            if ws.data_ptr() % 256:  # another allocator than torch's own
                ws = _new(nbytes + 256, torch.uint8, dev, stream, False)
                ws = ws[-ws.data_ptr() % 256:]
        else:
            ws, nbytes = _workspace(nbytes, torch.device("cuda", dev), workspace, stream)
    if stream is not None:
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(dev)
    else:
        handle = torch.cuda.current_stream(dev).cuda_stream
    args = (*args, ws.data_ptr() if ws is not None else None, nbytes, handle)
    if torch.cuda.current_device() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != GPTQ_OK:
        raise GPTQError(status, fn.__name__)


def dequant_gemm_adapters(x, packed, bits: int, cols: int, scales, zeros, groupsize: int, A, B,
                          scaling, index, g_idx=None, out=None, workspace=None, stream=None):
    """dequant_gemm (m x rows fp32) with each token's low-rank adapter:
    y_t += scaling[a] B[a] (A[a] x_t), a = index[t]; an index outside
    [0, count) adds nothing. A: count x rank x cols and B: count x rows x rank
    fp16, scaling: count fp32, index: m int32 (gptq_dequant_gemm_adapters)."""
    m, ldx, dev = _input(x, cols, "x")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev, g_idx)
    ad = _adapters(A, B, scaling, index, m, rows, cols, dev)
    out, ldy = _out_rows(out, m, rows, _f32, dev, stream)
    _launch(lib.gptq_dequant_gemm_adapters,
            (x.data_ptr(), m, cols, ldx, packed.data_ptr(), bits, rows, scales.data_ptr(),
             zeros.data_ptr(), groupsize, g_idx.data_ptr() if g_idx is not None else None, ad,
             out.data_ptr(), ldy),
            adapters_workspace_bytes(OP_FORWARD_ADAPTERS, m, rows, cols, ad.count, ad.rank), dev,
            workspace, stream)
    return out


def linear_forward_adapters(x, packed, bits: int, cols: int, scales, zeros, groupsize: int, A, B,
                            scaling, index, relu: bool = False, out=None, workspace=None,
                            stream=None):
    """linear_forward (m x rows fp16, many tokens) with each token's low-rank
    adapter, as dequant_gemm_adapters (gptq_linear_forward_adapters)."""
    m, ldx, dev = _input(x, cols, "x")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev)
    ad = _adapters(A, B, scaling, index, m, rows, cols, dev)
    out, ldy = _out_rows(out, m, rows, _f16, dev, stream)
    _launch(lib.gptq_linear_forward_adapters,
            (x.data_ptr(), m, cols, ldx, packed.data_ptr(), bits, rows, scales.data_ptr(),
             zeros.data_ptr(), groupsize, 1 if relu else 0, ad, out.data_ptr(), ldy),
            adapters_workspace_bytes(OP_FORWARD_ADAPTERS, m, rows, cols, ad.count, ad.rank), dev,
            workspace, stream)
    return out


def linear_backward(dy, packed, bits: int, cols: int, scales, zeros, groupsize: int, g_idx=None,
                    out=None, workspace=None, stream=None):
    """dx = dy W_hat (m x cols fp16) for dy m x rows fp16: the gradient
    through a stored layer (gptq_linear_backward without adapters)."""
    m, lddy, dev = _input(dy, None, "dy")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev, g_idx)
    _rows_of(dy, m, rows, _f16, dev, "dy")
    out, lddx = _out_rows(out, m, cols, _f16, dev, stream)
    _launch(lib.gptq_linear_backward,
            (dy.data_ptr(), m, rows, lddy, packed.data_ptr(), bits, cols, scales.data_ptr(),
             zeros.data_ptr(), groupsize, g_idx.data_ptr() if g_idx is not None else None, None,
             None, 0, out.data_ptr(), lddx, None, None),
            adapters_workspace_bytes(OP_BACKWARD, m, rows, cols), dev, workspace, stream)
    return out


def linear_backward_adapters(dy, x, packed, bits: int, cols: int, scales, zeros, groupsize: int, A,
                             B, scaling, index, g_idx=None, out=None, dA=None, dB=None,
                             workspace=None, stream=None):
    """(dx m x cols fp16, dA count x rank x cols fp32, dB count x rows x rank
    fp32) of the product with adapters for its input x and dy (m x rows fp16);
    where the forward product had relu, dy is zero where its output is 0
    (gptq_linear_backward)."""
    m, lddy, dev = _input(dy, None, "dy")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev, g_idx)
    _rows_of(dy, m, rows, _f16, dev, "dy")
    ldx = _rows_of(x, m, cols, _f16, dev, "x")
    ad = _adapters(A, B, scaling, index, m, rows, cols, dev)
    out, lddx = _out_rows(out, m, cols, _f16, dev, stream)
    dA = _out_exactly(dA, tuple(A.shape), _f32, dev, "dA", stream)
    dB = _out_exactly(dB, tuple(B.shape), _f32, dev, "dB", stream)
    _launch(lib.gptq_linear_backward,
            (dy.data_ptr(), m, rows, lddy, packed.data_ptr(), bits, cols, scales.data_ptr(),
             zeros.data_ptr(), groupsize, g_idx.data_ptr() if g_idx is not None else None, ad,
             x.data_ptr(), ldx, out.data_ptr(), lddx, dA.data_ptr(), dB.data_ptr()),
            adapters_workspace_bytes(OP_BACKWARD, m, rows, cols, ad.count, ad.rank), dev, workspace,
            stream)
    return out, dA, dB


def _head_entries(index, logits, m, dev):
    """The checks of labels (logits None: m) or of a teacher's entries (m x
    top); returns the shape of the entries' logits."""
    if logits is None:
        _exactly(index, (m,), _i32, dev, "target")
        return (m,)
    if index.dim() != 2:
        raise ValueError("top_index must be m x top")
    shape = (m, index.shape[1])
    _exactly(index, shape, _i32, dev, "top_index")
    _exactly(logits, shape, _f32, dev, "top_logits")
    return shape


def _temperature(t):
    t = float(t)
    if not 1e-30 < t < 1e30:
        raise ValueError("temperature must be positive")
    return t


def _head_forward(fn, h, layer, index, logits, more, loss, lse, zk, workspace, stream):
    packed, bits, cols, scales, zeros, groupsize = layer
    m, ldh, dev = _input(h, cols, "h")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev)
    shape = _head_entries(index, logits, m, dev)
    loss = _out_exactly(loss, (m,), _f32, dev, "loss", stream)
    lse = _out_exactly(lse, (m,), _f32, dev, "lse", stream)
    zk = _out_exactly(zk, shape, _f32, dev, "the entries' logits", stream)
    _launch(fn, (h.data_ptr(), m, cols, ldh, packed.data_ptr(), bits, rows, scales.data_ptr(),
                 zeros.data_ptr(), groupsize, index.data_ptr(), *more, loss.data_ptr(),
                 lse.data_ptr(), zk.data_ptr()),
            head_workspace_bytes(OP_HEAD_LOSS, m, rows, cols, shape[-1] if more else 1), dev,
            workspace, stream)
    return loss, lse, zk


def _head_backward(fn, h, layer, index, logits, more, lse, zk, dloss, out, workspace, stream):
    packed, bits, cols, scales, zeros, groupsize = layer
    m, ldh, dev = _input(h, cols, "h")
    rows, groupsize = _layer(packed, bits, cols, scales, zeros, groupsize, dev)
    shape = _head_entries(index, logits, m, dev)
    _exactly(lse, (m,), _f32, dev, "lse")
    _exactly(zk, shape, _f32, dev, "the entries' logits")
    _exactly(dloss, (m,), _f32, dev, "dloss")
    out, lddh = _out_rows(out, m, cols, _f16, dev, stream)
    _launch(fn, (h.data_ptr(), m, cols, ldh, packed.data_ptr(), bits, rows, scales.data_ptr(),
                 zeros.data_ptr(), groupsize, index.data_ptr(), *more, lse.data_ptr(),
                 zk.data_ptr(), dloss.data_ptr(), out.data_ptr(), lddh),
            head_workspace_bytes(OP_HEAD_BACKWARD, m, rows, cols, shape[-1] if more else 1), dev,
            workspace, stream)
    return out


def head_loss(h, packed, bits: int, cols: int, scales, zeros, groupsize: int, target, loss=None,
              lse=None, target_logit=None, workspace=None, stream=None):
    """Softmax cross entropy through a stored vocabulary projection, logits
    not kept: (loss, lse, target_logit), m fp32 each, for hidden states h
    (m x cols fp16) and labels target (m int32; outside [0, rows): the token
    takes no part). lse and target_logit are what head_loss_backward takes
    (gptq_head_loss)."""
    return _head_forward(lib.gptq_head_loss, h, (packed, bits, cols, scales, zeros, groupsize),
                         target, None, (), loss, lse, target_logit, workspace, stream)


def head_loss_backward(h, packed, bits: int, cols: int, scales, zeros, groupsize: int, target, lse,
                       target_logit, dloss, out=None, workspace=None, stream=None):
    """dh (m x cols fp16) of sum_t dloss[t] * loss[t] (gptq_head_loss_backward)."""
    return _head_backward(lib.gptq_head_loss_backward, h,
                          (packed, bits, cols, scales, zeros, groupsize), target, None, (), lse,
                          target_logit, dloss, out, workspace, stream)


def head_distill(h, packed, bits: int, cols: int, scales, zeros, groupsize: int, top_index,
                 top_logits, temperature: float = 1.0, loss=None, lse=None, student_logits=None,
                 workspace=None, stream=None):
    """Distillation from a teacher's largest logits through a stored
    vocabulary projection: (loss m, lse m, student_logits m x top, fp32) for
    top_index (int32) and top_logits (fp32), m x top; an index outside
    [0, rows) or a logit of -inf marks an entry that is not there
    (gptq_head_distill)."""
    t = _temperature(temperature)
    return _head_forward(lib.gptq_head_distill, h, (packed, bits, cols, scales, zeros, groupsize),
                         top_index, top_logits,
                         (top_logits.data_ptr(), top_logits.shape[-1], t), loss, lse,
                         student_logits, workspace, stream)


def head_distill_backward(h, packed, bits: int, cols: int, scales, zeros, groupsize: int,
                          top_index, top_logits, temperature, lse, student_logits, dloss, out=None,
                          workspace=None, stream=None):
    """dh (m x cols fp16) of sum_t dloss[t] * loss[t] of head_distill
    (gptq_head_distill_backward)."""
    t = _temperature(temperature)
    return _head_backward(lib.gptq_head_distill_backward, h,
                          (packed, bits, cols, scales, zeros, groupsize), top_index, top_logits,
                          (top_logits.data_ptr(), top_logits.shape[-1], t), lse, student_logits,
                          dloss, out, workspace, stream)
