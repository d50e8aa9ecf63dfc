"""Thin Python binding of libpq2 (ctypes).  Argument marshalling only: every
step of the path runs in the library's CUDA kernels.  torch supplies device
memory and streams.  There is no fallback: if libpq2.so is missing or a call
fails, an exception is raised.

Two levels:
  * ``lib()`` — the raw C functions with their exact C signatures (pointers
    as integers), used by tests that exercise the C ABI directly;
  * ``pq2_prepare``, ``pq2_quantize_act``, ``pq2_mmv``, ``pq2_mm``,
    ``pq2_debug_group_dots`` — the same names taking torch tensors, allocating
    outputs with torch when not given, and passing the current torch stream.

A call with ``stream`` runs on that stream, and what it allocates belongs to
it: a result is used on another stream after that one has waited for it, as with
any torch stream, and let go of when that use is done (or after
``record_stream``).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpq2.so")

PQ2_OK, PQ2_ERR_NULL, PQ2_ERR_SHAPE, PQ2_ERR_ALIGN, PQ2_ERR_DTYPE = 0, 1, 2, 3, 4
PQ2_ERR_ARCH, PQ2_ERR_LAUNCH, PQ2_ERR_TIMEOUT, PQ2_ERR_CUDA = 5, 6, 7, 8
PQ2_BF16, PQ2_F16, PQ2_F32, PQ2_I8 = 0, 1, 2, 3
PQ2_Q_ROWS, PQ2_Q_PLANES, PQ2_Q_F16, PQ2_Q_F8, PQ2_Q_MMV16 = 0, 1, 2, 3, 4
PQ2_DECODE_ADDXOR, PQ2_DECODE_PLANES = 0, 1
PQ2_PATH_MMV_ADDXOR, PQ2_PATH_MM, PQ2_PATH_MMV_PLANES, PQ2_PATH_MM_F8, PQ2_PATH_MMV_TC = \
    0, 1, 2, 3, 4
PQ2_MMV_OVERLAP_WEIGHTS, PQ2_MMV_INDEPENDENT = 1, 2
PQ2_STATIC_SCRATCH_BYTES = 1 << 20
PQ2_MAX_TOP = 32
PQ2_PREP_MAX_K = 32768
GROUP = 128



class CKvCache(ctypes.Structure):
    """pq2_kv_cache of include/pq2.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


# C signatures, mirroring include/pq2.h.
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "pq2_layout_version": (_I, []),
    "pq2_status_string": (ctypes.c_char_p, [_I]),
    "pq2_prepared_bytes": (_SZ, [_I64, _I64]),
    "pq2_prepare": (_I, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "pq2_quantize_act": (_I, [_P, _I, _I64, _I64, _I64, _P, _I, _P, _P, _P]),
    "pq2_mmv": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P]),
    "pq2_mmv_ex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _P]),
    "pq2_mmv_tc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P]),
    "pq2_linear_tensor_gemv": (_I, [_I64, _I64, _I64, _I]),
    "pq2_linear": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _I, _P, _SZ, _P, _P]),
    "pq2_linear_workspace_bytes": (_SZ, [_I64, _I64]),
    "pq2_linear_static": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _I, _P, _P]),
    "pq2_mmv_gated": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P]),
    "pq2_quantize_act_grouped": (_I, [_P, _I, _I64, _I64, _I64, _I, _P, _I, _P, _P, _P]),
    "pq2_ptq_prepare": (_I, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "pq2_ptq_linear_workspace_bytes": (_SZ, [_I64, _I64, _I]),
    "pq2_ptq_linear": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _P, _I, _P, _I, _P, _SZ, _P]),
    "pq2_ptq_mmv": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P]),
    "pq2_debug_ptq_dots": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    "pq2_mmv_grouped": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _P]),
    "pq2_debug_group_dots_grouped": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P]),
    "pq2_norm_hadamard_quantize": (_I, [_P, _P, _P, _P, _P, ctypes.c_float, _I64, _I64, _P,
                                        _P, _I, _P, _P, _P]),
    "pq2_linear_gated": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _I, _P, _SZ, _P, _P]),
    "pq2_mmv_decoder": (_I, [_I64]),
    "pq2_mm": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P]),
    "pq2_mm_f8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P]),
    "pq2_debug_group_dots": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P]),
    "pq2_mm_grouped": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P]),
    "pq2_mm_f8_grouped": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P]),
    "pq2_debug_mm_dots_grouped": (_I, [_P, _I, _P, _I64, _I64, _I64, _I, _P, _P, _P]),
    "pq2_linear_grouped_workspace_bytes": (_SZ, [_I64, _I64, _I]),
    "pq2_linear_grouped": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _P, _I, _P, _I, _P, _SZ, _P,
                                _P]),
    "pq2_w4_plane_bytes": (_SZ, [_I64, _I64, _I, _I]),
    "pq2_w4_prepare": (_I, [_P, _I64, _P, _P, _I64, _I64, _I, _P, _P]),
    "pq2_w4_mmv": (_I, [_P, _I, _I64, _I64, _I64, _I64, _I, _I, _P, _P, _I, _I, _P]),
    "pq2_token_logprobs": (_I, [_P, _I, _I64, _I64, _I64, ctypes.c_float, _P, _I64, _P, _P, _I,
                                _P, _P, _P]),
    "pq2_norm_gate_residual": (_I, [_P, _I64, _P, _I64, _I, _P, _P, _I64, _I64, ctypes.c_float,
                                    _P, ctypes.c_float, ctypes.c_float, _I64, _I64, _P, _P, _P]),
    "pq2_kv_store": (_I, [_P, _I64, _I64, _P, _I64, _I64, _I, _I64, _P, _P, _I64, _I64, _P, _P,
                          _I64, _P]),
    "pq2_kv_load": (_I, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _I, _I64, _P]),
    "pq2_attn_decode_workspace_bytes": (_SZ, [_I64] * 6),
    "pq2_attn_decode": (_I, [_P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _I64, _P,
                             ctypes.c_float, _P, _P, _P, _SZ, _P, _P]),
    "pq2_attn_prefill_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "pq2_attn_prefill": (_I, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I, _I64, _I64,
                              _I64, _I64, _I64, _P, _P, _I64, ctypes.c_float, _I, _P, _P, _P,
                              _SZ, _P, _P]),
    "pq2_mmv_geometry": (_I, [_I64, _I64, _I, _P, _P, _P, _P]),
    "pq2_debug_mmv_drop_arrival": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _P,
                                        _P]),
}

_lock = threading.Lock()
_lib = None


class Pq2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib().pq2_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")


def lib():
    """Load libpq2.so (it must have been built, see build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"libpq2.so not found at {LIB_PATH}; build it with "
                    "`python -m ternary_weight_int8_gb300.build`")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _lib = h
    return _lib


def _check(fn: str, status: int):
    if status != PQ2_OK:
        raise Pq2Error(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch.cuda.current_stream() builds a Stream object (3 us a call, as much as a
# whole small kernel); the raw handle is what the library takes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or _device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_device())


def _new(shape, dtype, device, stream):
    """A tensor that belongs to the call's stream: torch gives a block that the
    current stream has let go of to its next tensor at once, while kernels queued
    there may still use it, which another stream does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_DT = {torch.bfloat16: PQ2_BF16, torch.float16: PQ2_F16, torch.float32: PQ2_F32}


def prepared_bytes(N: int, K: int) -> int:
    return lib().pq2_prepared_bytes(N, K)


def pq2_prepare(raw: torch.Tensor, K: int, codes=None, scales=None, stream=None):
    """Raw blocks u8[N][>=K/128*34] (CUDA) -> (codes u8[N][K/4], scales fp16[N][K/128])."""
    N = raw.shape[0]
    if raw.dtype != torch.uint8 or raw.dim() != 2 or raw.stride(1) != 1:
        raise ValueError("raw must be a 2-D uint8 tensor with unit column stride")
    if codes is None:
        codes = _new((N, K // 4), torch.uint8, raw.device, stream)
    if scales is None:
        scales = _new((N, K // GROUP), torch.float16, raw.device, stream)
    _check("pq2_prepare", lib().pq2_prepare(_ptr(raw), raw.stride(0), N, K, _ptr(codes),
                                            _ptr(scales), _stream(stream)))
    return codes, scales


def pq2_quantize_act(x: torch.Tensor, layout: int = PQ2_Q_PLANES, q=None, sx=None,
                     qsum=None, want_qsum: bool = True, stream=None):
    """x[M][K] (bf16/f16/f32, CUDA, unit column stride) -> (q, sx, qsum)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    if q is None:
        q = q_buffer(M, K, layout, x.device, stream)
    if sx is None:
        sx = _new((M, K // GROUP), torch.float32, x.device, stream)
    if qsum is None and want_qsum:
        qsum = _new((M, K // GROUP), torch.int32, x.device, stream)
    _check("pq2_quantize_act",
           lib().pq2_quantize_act(_ptr(x), _DT[x.dtype], x.stride(0), M, K, _ptr(q), layout,
                                  _ptr(sx), _ptr(qsum), _stream(stream)))
    return q, sx, qsum


def pq2_mmv(q_planes, sx, qsum, codes, scales, y=None, out_dtype=torch.float32,
            decode=None, flags=0, status=None, stream=None):
    """Small-batch GEMV, M = 1..8: y[M][N] = sum_g dot * s_x * s_w."""
    M, K = q_planes.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_planes.device, stream)
    yd = _DT[y.dtype]
    args = (_ptr(q_planes), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales), _ptr(y), yd, M,
            N, K)
    if decode is None and not flags:
        st = lib().pq2_mmv(*args, _ptr(status), _stream(stream))
    else:
        dec = mmv_decoder(M) if decode is None else decode
        st = lib().pq2_mmv_ex(*args, dec, flags, _ptr(status), _stream(stream))
    _check("pq2_mmv", st)
    return y


def pq2_mmv_tc(q_mmv16, sx, qcorr, codes, scales, y=None, out_dtype=torch.float32, flags=0,
               status=None, stream=None):
    """Small-batch GEMV on the tensor-core path, M = 1..8, q from
    pq2_quantize_act(PQ2_Q_MMV16) and its corrections; same bits as pq2_mmv."""
    M, K = q_mmv16.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_mmv16.device, stream)
    _check("pq2_mmv_tc", lib().pq2_mmv_tc(_ptr(q_mmv16), _ptr(sx), _ptr(qcorr), _ptr(codes),
                                          _ptr(scales), _ptr(y), _DT[y.dtype], M, N, K, flags,
                                          _ptr(status), _stream(stream)))
    return y


def linear_workspace_bytes(M: int, K: int) -> int:
    return lib().pq2_linear_workspace_bytes(M, K)


def pq2_linear(x, codes, scales, y=None, out_dtype=torch.float32, workspace=None,
               status=None, stream=None):
    """Complete projection: quantise x, then the GEMV for M = 1..8 (streaming
    its weights while the quantisation runs) or the prefill GEMM from M = 9."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    wb = linear_workspace_bytes(M, K)
    if workspace is None:
        workspace = _new(wb, torch.uint8, x.device, stream)
    _check("pq2_linear", lib().pq2_linear(
        _ptr(x), _DT[x.dtype], x.stride(0), M, N, K, _ptr(codes), _ptr(scales), _ptr(y),
        _DT[y.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))
    return y


def pq2_quantize_act_grouped(x: torch.Tensor, act_group: int, layout: int = PQ2_Q_PLANES,
                             stream=None):
    """x[M][K] -> (q, sx [M][K/A], qsum [M][K/A]) with activation groups of A."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    q = q_buffer(M, K, layout, x.device, stream)
    sx = _new((M, K // act_group), torch.float32, x.device, stream)
    qsum = _new((M, K // act_group), torch.int32, x.device, stream)
    _check("pq2_quantize_act_grouped", lib().pq2_quantize_act_grouped(
        _ptr(x), _DT[x.dtype], x.stride(0), M, K, act_group, _ptr(q), layout, _ptr(sx),
        _ptr(qsum), _stream(stream)))
    return q, sx, qsum


def pq2_mmv_grouped(q_planes, sx, qsum, codes, scales, act_group: int, y=None,
                    out_dtype=torch.float32, flags=0, status=None, stream=None):
    """GEMV with activation groups of A (M = 1..4)."""
    M, K = q_planes.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_planes.device, stream)
    _check("pq2_mmv_grouped", lib().pq2_mmv_grouped(
        _ptr(q_planes), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales), _ptr(y), _DT[y.dtype],
        M, N, K, act_group, flags, _ptr(status), _stream(stream)))
    return y


def pq2_debug_group_dots_grouped(q_planes, qsum, codes, act_group: int, stream=None):
    """Exact partial dots [M][N][K/A] of the grouped GEMV's device code."""
    M, K = q_planes.shape
    N = codes.shape[0]
    dots = _new((M, N, K // act_group), torch.int32, q_planes.device, stream)
    _check("pq2_debug_group_dots_grouped", lib().pq2_debug_group_dots_grouped(
        _ptr(q_planes), _ptr(qsum), _ptr(codes), M, N, K, act_group, _ptr(dots), None,
        _stream(stream)))
    return dots


def pq2_ptq_prepare(raw: torch.Tensor, K: int, stream=None):
    """Raw PTQ1_0 rows u8[N][>= 28 K/128] (CUDA, unit column stride) ->
    (qs u8[N][24 K/128], side i32[N][K/128]: qh | d << 16)."""
    if raw.dim() != 2 or raw.stride(1) != 1 or raw.dtype != torch.uint8:
        raise ValueError("Expected a CUDA uint8 PTQ1_0 matrix")
    N = raw.shape[0]
    qs = _new((N, K // GROUP * 24), torch.uint8, raw.device, stream)
    side = _new((N, K // GROUP), torch.int32, raw.device, stream)
    _check("pq2_ptq_prepare", lib().pq2_ptq_prepare(_ptr(raw), raw.stride(0), N, K, _ptr(qs),
                                                     _ptr(side), _stream(stream)))
    return qs, side


def pq2_ptq_mmv(q_rows, sx, qsum, qs, side, act_group: int, y=None, out_dtype=torch.float32,
                flags=0, stream=None):
    """PTQ1_0 GEMV (M = 1..4) on row-layout grouped activations."""
    M, K = q_rows.shape
    N = qs.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_rows.device, stream)
    _check("pq2_ptq_mmv", lib().pq2_ptq_mmv(
        _ptr(q_rows), _ptr(sx), _ptr(qsum), _ptr(qs), _ptr(side), _ptr(y), _DT[y.dtype], M, N,
        K, act_group, flags, _stream(stream)))
    return y


def pq2_ptq_linear(x, qs, side, act_group: int, y=None, out_dtype=torch.float32, stream=None):
    """Complete PTQ1_0 projection (M = 1..4): grouped quantisation + GEMV."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    N = qs.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    nbytes = lib().pq2_ptq_linear_workspace_bytes(M, K, act_group)
    ws = _new(max(nbytes, 1), torch.uint8, x.device, stream)
    _check("pq2_ptq_linear", lib().pq2_ptq_linear(
        _ptr(x), _DT[x.dtype], x.stride(0), M, N, K, _ptr(qs), _ptr(side), act_group, _ptr(y),
        _DT[y.dtype], _ptr(ws), ws.numel(), _stream(stream)))
    return y


def pq2_debug_ptq_dots(q_rows, qsum, qs, side, act_group: int, stream=None):
    """Exact partial dots [M][N][K/A] of the PTQ1_0 GEMV's device code."""
    M, K = q_rows.shape
    N = qs.shape[0]
    dots = _new((M, N, K // act_group), torch.int32, q_rows.device, stream)
    _check("pq2_debug_ptq_dots", lib().pq2_debug_ptq_dots(
        _ptr(q_rows), _ptr(qsum), _ptr(qs), _ptr(side), M, N, K, act_group, _ptr(dots),
        _stream(stream)))
    return dots


def pq2_mmv_gated(q_planes, sx, qsum, codes, scales, out=None, out_dtype=torch.float32,
                  flags=0, status=None, stream=None):
    """Gate/up GEMV with its gated activation, M = 1..8: codes/scales hold N
    rows (gate rows, then up rows); out[M][N/2] = silu(gate) * up."""
    M, K = q_planes.shape
    N = codes.shape[0]
    if out is None:
        out = _new((M, N // 2), out_dtype, q_planes.device, stream)
    _check("pq2_mmv_gated", lib().pq2_mmv_gated(
        _ptr(q_planes), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales), _ptr(out),
        _DT[out.dtype], M, N, K, flags, _ptr(status), _stream(stream)))
    return out


def pq2_linear_gated(x, codes, scales, out=None, out_dtype=torch.float32, workspace=None,
                     status=None, stream=None):
    """Complete gated call for M = 1..8: quantise x, then pq2_mmv_gated."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    N = codes.shape[0]
    if out is None:
        out = _new((M, N // 2), out_dtype, x.device, stream)
    if workspace is None:
        workspace = _new(linear_workspace_bytes(M, K), torch.uint8, x.device, stream)
    _check("pq2_linear_gated", lib().pq2_linear_gated(
        _ptr(x), _DT[x.dtype], x.stride(0), M, N, K, _ptr(codes), _ptr(scales), _ptr(out),
        _DT[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))
    return out


def pq2_norm_hadamard_quantize(x, w, sign, eps, residual=None, layout: int = PQ2_Q_PLANES,
                               want_norm=False, want_residual=False, stream=None):
    """x bf16 [M][K] (CUDA), norm weight w bf16 [K], sign int8 [K] (+-1) ->
    (q, sx, qsum, norm_out or None, residual_out or None): RMSNorm, signs,
    1024-point Walsh-Hadamard and group-128 quantisation in one kernel."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 tensor")
    M, K = x.shape
    q = q_buffer(M, K, layout, x.device, stream)
    sx = _new((M, K // GROUP), torch.float32, x.device, stream)
    qsum = _new((M, K // GROUP), torch.int32, x.device, stream)
    norm = _new(x.shape, x.dtype, x.device, stream) if want_norm else None
    rout = _new(x.shape, x.dtype, x.device, stream) if want_residual else None
    _check("pq2_norm_hadamard_quantize", lib().pq2_norm_hadamard_quantize(
        _ptr(x), _ptr(residual), _ptr(rout), _ptr(w), _ptr(sign), float(eps), M, K,
        _ptr(norm), _ptr(q), layout, _ptr(sx), _ptr(qsum), _stream(stream)))
    return q, sx, qsum, norm, rout


def q_buffer(M: int, K: int, layout: int, device, stream=None):
    """Output buffer of the quantiser for `layout`: fp16 [M][K] (PQ2_Q_F16,
    PQ2_Q_MMV16), uint8 [M][2K] (the two e4m3 planes of PQ2_Q_F8) or int8
    [M][K]."""
    if layout in (PQ2_Q_F16, PQ2_Q_MMV16):
        return _new((M, K), torch.float16, device, stream)
    if layout == PQ2_Q_F8:
        return _new((M, 2 * K), torch.uint8, device, stream)
    return _new((M, K), torch.int8, device, stream)


def pq2_mm_f8(q_f8, sx, qsum, codes, scales, y=None, out_dtype=torch.float32, status=None,
              stream=None):
    """Prefill matmul (M >= 16; any M >= 1) on the 8-bit tcgen05 path (q from PQ2_Q_F8)."""
    M, K = q_f8.shape[0], q_f8.shape[1] // 2
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_f8.device, stream)
    _check("pq2_mm_f8", lib().pq2_mm_f8(_ptr(q_f8), _ptr(sx), _ptr(qsum), _ptr(codes),
                                        _ptr(scales), _ptr(y), _DT[y.dtype], M, N, K,
                                        _ptr(status), _stream(stream)))
    return y


def pq2_mm(q_f16, sx, qsum, codes, scales, y=None, out_dtype=torch.float32, status=None,
           stream=None):
    """Prefill matmul (M >= 16; any M >= 1) on tcgen05 tensor cores."""
    M, K = q_f16.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_f16.device, stream)
    _check("pq2_mm", lib().pq2_mm(_ptr(q_f16), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales),
                                  _ptr(y), _DT[y.dtype], M, N, K, _ptr(status),
                                  _stream(stream)))
    return y


def pq2_debug_group_dots(q, codes, path: int, qsum=None, dots=None, status=None,
                         stream=None):
    """Exact int32 group dots [M][N][K/128] from the kernels' own decode/dot code."""
    M, K = q.shape
    if path == PQ2_PATH_MM_F8:
        K //= 2
    N = codes.shape[0]
    if dots is None:
        dots = _new((M, N, K // GROUP), torch.int32, q.device, stream)
    _check("pq2_debug_group_dots",
           lib().pq2_debug_group_dots(_ptr(q), _ptr(qsum), _ptr(codes), M, N, K, path,
                                      _ptr(dots), _ptr(status), _stream(stream)))
    return dots


def pq2_mm_grouped(q_f16, sx, qsum, codes, scales, act_group: int, y=None,
                   out_dtype=torch.float32, status=None, stream=None):
    """Prefill matmul with activation groups of A (q from
    pq2_quantize_act_grouped, PQ2_Q_F16)."""
    M, K = q_f16.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_f16.device, stream)
    _check("pq2_mm_grouped", lib().pq2_mm_grouped(
        _ptr(q_f16), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales), _ptr(y), _DT[y.dtype],
        M, N, K, act_group, _ptr(status), _stream(stream)))
    return y


def pq2_mm_f8_grouped(q_f8, sx, qsum, codes, scales, act_group: int, y=None,
                      out_dtype=torch.float32, status=None, stream=None):
    """pq2_mm_grouped on the 8-bit tensor path (q PQ2_Q_F8)."""
    M, K = q_f8.shape[0], q_f8.shape[1] // 2
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, q_f8.device, stream)
    _check("pq2_mm_f8_grouped", lib().pq2_mm_f8_grouped(
        _ptr(q_f8), _ptr(sx), _ptr(qsum), _ptr(codes), _ptr(scales), _ptr(y), _DT[y.dtype],
        M, N, K, act_group, _ptr(status), _stream(stream)))
    return y


def pq2_debug_mm_dots_grouped(q, codes, path: int, act_group: int, dots=None, status=None,
                              stream=None):
    """Exact partial dots [M][N][K/A] of the grouped prefill kernels."""
    M, K = q.shape
    if path == PQ2_PATH_MM_F8:
        K //= 2
    N = codes.shape[0]
    if dots is None:
        dots = _new((M, N, K // act_group), torch.int32, q.device, stream)
    _check("pq2_debug_mm_dots_grouped", lib().pq2_debug_mm_dots_grouped(
        _ptr(q), path, _ptr(codes), M, N, K, act_group, _ptr(dots), _ptr(status),
        _stream(stream)))
    return dots


def linear_grouped_workspace_bytes(M: int, K: int, act_group: int) -> int:
    return lib().pq2_linear_grouped_workspace_bytes(M, K, act_group)


def pq2_linear_grouped(x, codes, scales, act_group: int, y=None, out_dtype=torch.float32,
                       workspace=None, status=None, stream=None):
    """Complete projection with activation groups of A: the grouped quantiser,
    then the grouped GEMV (M = 1..8) or the grouped prefill GEMM (M >= 9)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    if workspace is None:
        workspace = _new(linear_grouped_workspace_bytes(M, K, act_group), torch.uint8, x.device,
                         stream)
    _check("pq2_linear_grouped", lib().pq2_linear_grouped(
        _ptr(x), _DT[x.dtype], x.stride(0), M, N, K, _ptr(codes), _ptr(scales), act_group,
        _ptr(y), _DT[y.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))
    return y


def _on_device(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda and not t.is_pinned():
            raise ValueError("Expected CUDA tensors (or pinned host memory)")


def _check_plane(plane):
    # The kernels take its bytes from the first one on.
    if plane.dtype != torch.uint8 or not plane.is_contiguous():
        raise ValueError("plane must be a contiguous uint8 tensor")


def pq2_w4_prepare(codes, scales, zeros=None, group: int = 128, plane=None, stream=None):
    """4-bit codes u8[N][K/2] (column 2j in the low half of byte j), fp16
    scales [N][K/group] and zero points u8[N][K/group] (None: 8) -> the plane
    u8 that pq2_w4_mmv streams."""
    if codes.dim() != 2 or codes.dtype != torch.uint8 or codes.stride(1) != 1:
        raise ValueError("codes must be a 2-D uint8 tensor with unit column stride")
    if plane is not None:
        _check_plane(plane)
    if group < 1:
        raise Pq2Error("pq2_w4_prepare", PQ2_ERR_SHAPE)
    _on_device(codes, scales, zeros, plane)
    N, K = codes.shape[0], 2 * codes.shape[1]
    for t, dt, what in ((scales, torch.float16, "fp16 scales"), (zeros, torch.uint8, "uint8 zeros")):
        if t is not None and (t.dtype != dt or t.shape != (N, K // group)
                              or not t.is_contiguous()):
            raise ValueError(f"Expected contiguous {what} of shape [N][K / group]")
    nbytes = lib().pq2_w4_plane_bytes(N, K, group, int(zeros is not None))
    if plane is None:
        plane = _new(max(nbytes, 1), torch.uint8, codes.device, stream)
    elif plane.numel() < nbytes:
        raise Pq2Error("pq2_w4_prepare", PQ2_ERR_SHAPE)
    _check("pq2_w4_prepare", lib().pq2_w4_prepare(
        _ptr(codes), codes.stride(0), _ptr(scales), _ptr(zeros), N, K, group, _ptr(plane),
        _stream(stream)))
    return plane


_w4_bytes = {}


def _dtype_of(t):
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"Expected a bfloat16, float16 or float32 tensor, not {t.dtype}")
    return code


def _check_out(t, shape, dtype=None):
    if t.shape != shape or not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"Expected a contiguous output buffer of shape {tuple(shape)}")


def pq2_w4_mmv(x, plane, N: int, group: int = 128, zeros: bool = False, y=None,
               out_dtype=torch.float32, flags=0, stream=None):
    """y[M][N] = x W^T for M = 1..32 on a plane of N rows from pq2_w4_prepare
    (group and zeros as there)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    _check_plane(plane)
    M, K = x.shape
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    else:
        _check_out(y, (M, N))
    x_dtype, y_dtype = _dtype_of(x), _dtype_of(y)
    _on_device(x, plane, y)
    key = (N, K, group, zeros)
    if key not in _w4_bytes:
        _w4_bytes[key] = lib().pq2_w4_plane_bytes(N, K, group, int(zeros))
    if plane.numel() < _w4_bytes[key]:
        raise Pq2Error("pq2_w4_mmv", PQ2_ERR_SHAPE)
    _check("pq2_w4_mmv", lib().pq2_w4_mmv(
        _ptr(x), x_dtype, x.stride(0), M, N, K, group, int(zeros), _ptr(plane), _ptr(y),
        y_dtype, flags, _stream(stream)))
    return y


def pq2_token_logprobs(logits, tokens=None, k: int = 0, scale: float = 1.0, entropy: bool = True,
                       out=None, stream=None):
    """logits[M][V], tokens int64 [M][T] or [M] (None: none) ->
    (token_logprobs [M][T], entropy [M] or None, top_ids int64 [M][k],
    top_logprobs [M][k]); `out` is that tuple of buffers."""
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit column stride")
    dtype = _dtype_of(logits)
    M, V = logits.shape
    if tokens is not None and (tokens.dtype != torch.int64 or not tokens.is_contiguous()
                               or tokens.shape[0] != M):
        raise ValueError("Expected contiguous int64 tokens with a row per row of logits")
    _on_device(logits, tokens)
    T = 0 if tokens is None or not M else tokens.numel() // M
    if out is None:
        dev = logits.device
        out = (_new((M, T), torch.float32, dev, stream),
               _new((M,), torch.float32, dev, stream) if entropy else None,
               _new((M, k), torch.int64, dev, stream),
               _new((M, k), torch.float32, dev, stream))
    else:
        _on_device(*out)
        _check_out(out[0], (M, T), torch.float32)
        if out[1] is not None:
            _check_out(out[1], (M,), torch.float32)
        _check_out(out[2], (M, k), torch.int64)
        _check_out(out[3], (M, k), torch.float32)
    _check("pq2_token_logprobs", lib().pq2_token_logprobs(
        _ptr(logits), dtype, logits.stride(0), M, V, scale, _ptr(tokens), T,
        _ptr(out[0]) if T else None, _ptr(out[1]), k, _ptr(out[2]) if k else None,
        _ptr(out[3]) if k else None, _stream(stream)))
    return out


def pq2_norm_gate_residual(z, h, w_pre, w_post=None, gate=None, rows_per_gate: int = 1,
                           alpha: float = 1.0, eps: float = 1e-6, w_offset: float = 0.0,
                           h_out=None, n_out=None, stream=None):
    """The norms around a block with its gate and residual scale:
    h' = h + alpha * gate * norm(z, w_post), n = norm(h', w_pre) ->
    (h_out, n_out).  z None: the plain norm of h (h_out None); w_pre None: no
    n_out.  All tensors have h's type."""
    dtype = h.dtype
    if h.dim() != 2 or h.stride(1) != 1:
        raise ValueError("h must be 2-D with unit column stride")
    code = _dtype_of(h)
    M, K = shape = h.shape
    ldz = ldg = 0
    if z is not None:
        if z.shape != shape or z.dtype != dtype or z.stride(1) != 1:
            raise ValueError("z must have h's shape and type and unit column stride")
        ldz = z.stride(0)
    if gate is not None:
        if gate.dim() != 2 or gate.shape[1] != K or gate.shape[0] * rows_per_gate < M or \
                gate.dtype != dtype or gate.stride(1) != 1:
            raise ValueError("gate must have h's type, K columns with unit stride and a row per "
                             "rows_per_gate rows of h")
        ldg = gate.stride(0)
    if w_pre is not None and (w_pre.numel() != K or w_pre.dtype != dtype
                              or not w_pre.is_contiguous()) or \
            w_post is not None and (w_post.numel() != K or w_post.dtype != dtype
                                    or not w_post.is_contiguous()):
        raise ValueError("the norm weights must be contiguous [K] of h's type")
    _on_device(z, h, w_pre, w_post, gate, h_out, n_out)
    if h_out is not None:
        _check_out(h_out, shape, dtype)
    elif z is not None:
        h_out = _new((M, K), dtype, h.device, stream)
    if n_out is not None:
        _check_out(n_out, shape, dtype)
    elif w_pre is not None:
        n_out = _new((M, K), dtype, h.device, stream)
    _check("pq2_norm_gate_residual", lib().pq2_norm_gate_residual(
        _ptr(z), ldz, _ptr(h), h.stride(0), code, _ptr(w_post), _ptr(gate), ldg,
        rows_per_gate, alpha, _ptr(w_pre), w_offset, eps, M, K, _ptr(h_out), _ptr(n_out),
        _stream(stream)))
    return h_out, n_out


class KVCache(NamedTuple):
    """The pages of a key-value cache: k and v [pages][heads][page_size][dim]
    (bfloat16, float16 or int8; any equal strides, unit for dim), and for int8
    their scales fp32 [pages][heads][page_size]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None


def kv_cache(pages: int, heads: int, page_size: int, dim: int, dtype=torch.int8, device="cuda"):
    """A new, empty KVCache."""
    shape = (pages, heads, page_size, dim)
    if dtype not in _CACHE_DT:
        raise ValueError("Expected an int8, float16 or bfloat16 cache")
    scales = [torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)] \
        if dtype == torch.int8 else (None, None)
    return KVCache(torch.zeros(shape, dtype=dtype, device=device),
                   torch.zeros(shape, dtype=dtype, device=device), *scales)


_CACHE_DT = {torch.bfloat16: PQ2_BF16, torch.float16: PQ2_F16, torch.int8: PQ2_I8}


def _strides(t):
    """Strides for the C ABI: those of dimensions with one element are never
    walked, and torch leaves anything in them."""
    return [s if n > 1 else 0 for n, s in zip(t.shape, t.stride())]


# pq2_kv_cache as bytes: cheaper to make than a ctypes structure.
_KV_CACHE = struct.Struct("@PPPPiqqqqqqq")


def _c_cache(cache):
    """(pq2_kv_cache, heads, dim) of a KVCache, after the checks."""
    k, v, ks, vs = cache
    shape, st, code = k.shape, k.stride(), _CACHE_DT.get(k.dtype)
    if code is None or len(shape) != 4 or v.shape != shape or v.dtype != k.dtype or \
            st[3] != 1 or (v.stride() != st and (v.stride(3) != 1 or _strides(k) != _strides(v))):
        raise ValueError("a cache's k and v must be 4-D int8, float16 or bfloat16 tensors of one "
                         "shape and strides, with unit stride in dim")
    if code != PQ2_I8:
        if ks is not None or vs is not None:
            raise ValueError("an int8 cache has scales, others have none")
        sides = 0, 0
    else:
        if ks is None or vs is None:
            raise ValueError("an int8 cache has scales, others have none")
        for t in (ks, vs):
            if t.dtype != torch.float32 or t.shape != shape[:3] or not t.is_contiguous():
                raise ValueError("the scales must be contiguous float32 [pages][heads][page_size]")
        sides = ks.data_ptr(), vs.data_ptr()
    if 1 in shape:
        st = _strides(k)
    return _KV_CACHE.pack(k.data_ptr(), v.data_ptr(), *sides, code, *shape, *st[:3]), shape[1], \
        shape[3]


def _check_ints(t, what, n=None):
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or \
            n is not None and t.shape[0] != n:
        raise ValueError(f"{what} must be contiguous int32" + (f" [{n}]" if n is not None else ""))


def _check_table(table, lens, cu=None):
    """(B, row stride, width) of a page table, after the checks of a batch."""
    shape = table.shape
    if len(shape) != 2 or table.dtype != torch.int32 or (table.stride(1) != 1 and shape[1] > 1):
        raise ValueError("table must be 2-D int32 with unit column stride")
    B, width = shape
    _check_ints(lens, "lens", B)
    if cu is not None:
        _check_ints(cu, "cu", B + 1)
    return B, table.stride(0) if B > 1 else width, width


def _on_one_device(first, *others):
    """CUDA tensors of one device, the current one (whose stream is used)."""
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            device = -1
    if device < 0:
        raise ValueError("Expected CUDA tensors of one device")
    if device != (torch.cuda.current_device() if _device is None else _device()):
        raise ValueError("the tensors' device must be the current device")


def pq2_kv_store(k, v, cache: KVCache, table, lens, cu=None, stream=None):
    """Writes the newest tokens' keys and values k, v [tokens][heads][dim] into
    the cache: sequence b's rows cu[b]..cu[b+1] (cu None: the rows split evenly)
    are its last positions before lens[b]; page table[b][p // page_size] holds
    position p."""
    c, heads, dim = _c_cache(cache)
    shape, ks, vs = k.shape, k.stride(), v.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or v.shape != shape or \
            v.dtype != k.dtype or ks[2] != 1 or vs[2] != 1:
        raise ValueError("k and v must be [tokens][heads][dim] of one type, with the cache's heads "
                         "and dim and unit stride in dim")
    dtype = _dtype_of(k)
    B, stride, width = _check_table(table, lens, cu)
    _on_one_device(k, v, *cache, table, lens, cu)
    _check("pq2_kv_store", lib().pq2_kv_store(
        k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], dtype, shape[0], c,
        table.data_ptr(), stride, width, _ptr(cu), lens.data_ptr(), B, _stream(stream)))


def pq2_kv_load(cache: KVCache, table, lens, cu=None, tokens=None, out=None,
                out_dtype=torch.bfloat16, stream=None):
    """The last cu[b+1] - cu[b] positions of each sequence, read back and packed
    -> (k, v) [tokens][heads][dim]; `out` is that pair of buffers, else `tokens`
    gives their rows."""
    c, heads, dim = _c_cache(cache)
    B, stride, width = _check_table(table, lens, cu)
    if out is None:
        if tokens is None:
            raise ValueError("either out or tokens must be given")
        out = [_new((tokens, heads, dim), out_dtype, cache.k.device, stream) for _ in range(2)]
    k, v = out
    shape = (k.shape[0] if tokens is None else tokens, heads, dim)
    dtype = _dtype_of(k)
    _check_out(k, shape)
    _check_out(v, shape, k.dtype)
    _on_one_device(k, v, *cache, table, lens, cu)
    _check("pq2_kv_load", lib().pq2_kv_load(
        c, table.data_ptr(), stride, width, _ptr(cu), lens.data_ptr(), B, k.data_ptr(),
        v.data_ptr(), dtype, shape[0], _stream(stream)))
    return k, v


_attn_bytes = {}


def _workspace(nbytes, like, stream):
    return _new(nbytes, torch.uint8, like.device, stream)


_kept = threading.local()  # .by: {(device, stream): a workspace of this thread's calls on it}
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)


def _kept_workspace(nbytes, like, stream):
    """pq2_attn_decode's: a few MB, kept, as allocating them costs more than the
    launch.  A thread's calls on one stream follow one another; another thread's
    may come between a call's two kernels.  A captured graph may be replayed
    anywhere, beside other graphs: it gets one of its own."""
    if stream is not None or not like.is_cuda or _capturing is None or _capturing():
        return _workspace(nbytes, like, stream)
    by = _kept.__dict__.setdefault("by", {})
    key = like.device, _stream(None)
    w = by.get(key)
    if w is None or w.numel() < nbytes:
        w = by[key] = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return w


def _attn_outputs(q, out, lse, stream):
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"Expected a bfloat16 or float16 tensor, not {q.dtype}")
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    else:
        _check_out(out, q.shape, q.dtype)
    if lse is not None:
        _check_out(lse, q.shape[:-1], torch.float32)
    return out


def pq2_attn_decode(q, cache: KVCache, table, lens, scale=None, out=None, lse=None,
                    workspace=None, status=None, stream=None):
    """Attention of the newest token(s) of each sequence over its cache, which
    holds their keys and values already: q [B][heads][dim] or [B][T][heads][dim]
    -> out of q's shape.  Token t of T sees the positions before
    lens[b] - T + t + 1.  scale: 1 / sqrt(dim) if None; lse: a float32 buffer of
    q.shape[:-1] for the rows' log-sum-exp; workspace: if None, one of up to 11 MB
    that is kept per thread and stream while the process lives (a captured call, or
    one with stream, gets its own)."""
    L = lib()
    c, kv_heads, dim = _c_cache(cache)
    shape, st = q.shape, q.stride()
    if len(shape) not in (3, 4) or st[-1] != 1 or shape[-1] != dim:
        raise ValueError("q must be [B][heads][dim] or [B][T][heads][dim] with unit stride in dim")
    if 1 in shape:
        st = _strides(q)
    B, stride, width = _check_table(table, lens)
    if shape[0] != B:
        raise ValueError("q must have a row per row of the table")
    out = _attn_outputs(q, out, lse, stream)
    T, T_stride = (1, 0) if len(shape) == 3 else (shape[1], st[1])
    if cache.k.dtype not in (q.dtype, torch.int8):
        raise ValueError("the cache must have q's type, or int8")
    if workspace is None:
        key = (B, T, shape[-2], kv_heads, dim, width * cache.k.shape[2])
        nbytes = _attn_bytes.get(key)
        if nbytes is None:
            if len(_attn_bytes) > 4096:
                _attn_bytes.clear()
            nbytes = _attn_bytes[key] = L.pq2_attn_decode_workspace_bytes(*key)
        if nbytes:
            workspace = _kept_workspace(nbytes, q, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _on_one_device(q, *cache, table, lens, out, lse, workspace, status)
    _check("pq2_attn_decode", L.pq2_attn_decode(
        q.data_ptr(), _DT[q.dtype], st[0], T_stride, st[-2], B, T, shape[-2], c,
        table.data_ptr(), stride, width, lens.data_ptr(), dim ** -0.5 if scale is None else scale,
        out.data_ptr(), _ptr(lse), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))
    return out


def pq2_attn_prefill(q, k, v, cu_q, cu_k=None, scale=None, causal: bool = True, out=None,
                     lse=None, workspace=None, status=None, stream=None):
    """Attention over packed sequences: rows cu_q[b]..cu_q[b+1] of q
    [rows][heads][dim] attend rows cu_k[b]..cu_k[b+1] (None: the same) of k and
    v [rows][key heads][dim]; causal counts both from their ends.  scale and lse
    as in pq2_attn_decode."""
    q_shape, k_shape, qs, ks, vs = q.shape, k.shape, q.stride(), k.stride(), v.stride()
    if len(q_shape) != 3 or len(k_shape) != 3 or q_shape[2] != k_shape[2] or \
            v.shape != k_shape or qs[2] != 1 or ks[2] != 1 or vs[2] != 1:
        raise ValueError("q, k and v must be [rows][heads][dim] with unit stride in dim, k and v of "
                         "one shape and q's dim")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must have q's type")
    cu_k = cu_q if cu_k is None else cu_k
    _check_ints(cu_q, "cu_q")
    _check_ints(cu_k, "cu_k", cu_q.shape[0])
    out = _attn_outputs(q, out, lse, stream)
    rows, heads, dim = q_shape
    keys, kv_heads, B = k_shape[0], k_shape[1], cu_q.shape[0] - 1
    if 1 in q_shape or 1 in k_shape:
        qs, ks, vs = _strides(q), _strides(k), _strides(v)
    if workspace is None:
        nbytes = lib().pq2_attn_prefill_workspace_bytes(B, rows, keys, heads, kv_heads, dim)
        if nbytes:
            workspace = _workspace(nbytes, q, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _on_one_device(q, k, v, cu_q, cu_k, out, lse, workspace, status)
    _check("pq2_attn_prefill", lib().pq2_attn_prefill(
        _ptr(q), qs[0], qs[1], _ptr(k), ks[0], ks[1], _ptr(v), vs[0], vs[1], _DT[q.dtype], rows,
        keys, heads, kv_heads, dim, _ptr(cu_q), _ptr(cu_k), B,
        dim ** -0.5 if scale is None else scale, int(causal), _ptr(out), _ptr(lse),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))
    return out


def mmv_geometry(N: int, K: int, sm_count: int):
    """(ctas, threads, splits, rows_max) of pq2_mmv for (N, K) — host only."""
    out = [ctypes.c_int() for _ in range(4)]
    _check("pq2_mmv_geometry", lib().pq2_mmv_geometry(
        N, K, sm_count, *[ctypes.addressof(o) for o in out]))
    return tuple(o.value for o in out)


def mmv_decoder(M: int) -> int:
    return lib().pq2_mmv_decoder(M)


def linear(x, codes, scales, out_dtype=torch.float32, stream=None):
    """The complete projection: pq2_linear (the GEMV for M <= 8, the
    prefill GEMM from M = 9)."""
    return pq2_linear(x, codes, scales, out_dtype=out_dtype, stream=stream)
