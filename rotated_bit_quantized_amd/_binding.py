"""ctypes binding of liboq (include/oq.h): argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
PyTorch tensors on a HIP device (PyTorch provides device memory and the
current stream); outputs that are not supplied are allocated with
``torch.empty``.  All arithmetic runs in the library's HIP kernels; there is
no other code path.  A non-zero status raises :class:`OQError`.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liboq.so")

OQ_OK, OQ_ERR_INVALID_ARG, OQ_ERR_UNSUPPORTED, OQ_ERR_ALIGNMENT, OQ_ERR_WORKSPACE, OQ_ERR_HIP = range(6)
OQ_ROT_RPBH, OQ_ROT_DENSE32, OQ_ROT_KRON = 1, 2, 3
OQ_A8, OQ_A6, OQ_A4, OQ_MXFP4 = 8, 6, 4, 0x104
OQ_W4, OQ_W_MXFP4 = 4, 0x104
OQ_OP_GEMM_W4A8, OQ_OP_GEMM_W4A4, OQ_OP_LINEAR, OQ_OP_GEMM_LM = 1, 2, 3, 4
OQ_TILED = 0x10000
OQ_SCALE_PCTL = 0x20000
OQ_F32, OQ_BF16 = 1, 2
OQ_SCORE_SOFTMAX, OQ_SCORE_SIGMOID = 1, 2
OQ_ACT_NONE, OQ_ACT_SWIGLU = 0, 1
OQ_NORM_RMS, OQ_NORM_LAYER = 1, 2


class OQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[oq error {code}] {msg}")
        self.code = code


class oq_rot(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("block", ctypes.c_int32),
        ("rounds", ctypes.c_int32),
        ("perm", ctypes.c_void_p),
        ("signs", ctypes.c_void_p),
        ("mats", ctypes.c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"liboq.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    f32 = ctypes.c_float
    sig = {
        "oq_last_error": ([], ctypes.c_char_p),
        "oq_center": ([vp, i64, i32, i64, vp, i64, vp, vp], ctypes.c_int),
        "oq_rotate": ([vp, vp, i64, i64, ctypes.c_int, vp, vp, i64, vp], ctypes.c_int),
        "oq_quant_act": ([vp, i64, i32, i64, vp, ctypes.c_int, ctypes.c_int, vp, i64, vp, vp, vp, vp], ctypes.c_int),
        "oq_quant_weight": ([vp, i32, i32, i64, vp, ctypes.c_int, i32, vp, vp, vp, vp], ctypes.c_int),
        "oq_gemm_w4a8": ([vp, i64, vp, i64, i32, vp, vp, i32, i32, vp, vp, vp, vp, i64, vp, sz, vp], ctypes.c_int),
        "oq_gemm_w4a4": ([ctypes.c_int, vp, i64, vp, i64, i32, vp, vp, i32, i32, vp, vp, vp, vp, i64, vp, sz, vp], ctypes.c_int),
        "oq_linear_fused": ([vp, i64, i32, i64, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, vp, vp, vp, i64, vp, sz, vp], ctypes.c_int),
        "oq_probe_mfma": ([ctypes.c_int, i32, vp, ctypes.POINTER(ctypes.c_double), vp], ctypes.c_int),
        "oq_probe_sink_elems": ([], sz),
        "oq_linear_fused_noalloc": ([vp, i64, i32, i64, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, vp, vp, vp,
                                     i64, vp], ctypes.c_int),
        "oq_workspace_bytes": ([ctypes.c_int, i64, i32, i32, ctypes.c_int], sz),
        "oq_tiled_bytes": ([i64, i32], sz),
        "oq_prepack_w4": ([vp, vp, i32, i32, i32, vp, vp, vp], ctypes.c_int),
        "oq_tiled_mx_bytes": ([i64, i32], sz),
        "oq_prepack_mx": ([vp, vp, i32, i32, vp, vp, vp], ctypes.c_int),
        "oq_lloyd_max_levels": ([i32, i32, vp], ctypes.c_int),
        "oq_lloyd_max_tables": ([i32, i32, vp, vp], ctypes.c_int),
        "oq_tiled_f16_bytes": ([i64, i32], sz),
        "oq_quant_act_lm": ([vp, i64, i32, i64, vp, ctypes.c_int, i32, ctypes.c_int, vp, vp, vp, i64, vp, vp, vp],
                            ctypes.c_int),
        "oq_prepack_w16": ([vp, vp, i32, i32, i32, vp, vp], ctypes.c_int),
        "oq_gemm_lm": ([i32, ctypes.c_int, vp, i64, vp, i64, i32, vp, vp, i32, vp, vp, vp, vp, i64, vp, sz, vp],
                       ctypes.c_int),
        "oq_quant_weight_asym": ([vp, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp], ctypes.c_int),
        "oq_prepack_w4_asym": ([vp, vp, vp, i32, i32, i32, vp, vp, vp, vp], ctypes.c_int),
        "oq_quant_act_gsum": ([vp, i64, i32, i64, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp], ctypes.c_int),
        "oq_gemm_w4a4_asym": ([ctypes.c_int, vp, vp, vp, i64, i32, vp, vp, vp, i32, vp, vp, vp, vp, i64, vp],
                              ctypes.c_int),
        "oq_kron_plan": ([i32, vp, vp, vp], ctypes.c_int),
        "oq_quant_weight_w8": ([vp, i32, i32, i64, vp, vp, i64, vp, vp, vp], ctypes.c_int),
        "oq_gemm_w8a8": ([vp, i64, vp, i64, i32, vp, i64, vp, i32, vp, vp, vp, vp, i64, vp], ctypes.c_int),
        "oq_qk_norm_rope": ([vp, i64, i64, i32, vp, i64, i64, i32, i64, i32, vp, vp, f32, vp, vp, vp, i64, i64, vp, i64,
                             i64, vp], ctypes.c_int),
        "oq_kv_append": ([vp, i64, i64, vp, i64, i64, i64, vp, f32, vp, vp, vp, vp, vp], ctypes.c_int),
        "oq_attn_prefix": ([vp, i64, i64, i32, i32, i32, vp, vp, i32, vp, i32, vp, f32, vp, i64, i64, vp, vp, sz, vp],
                           ctypes.c_int),
        "oq_attn_prefix_ws_bytes": ([i32, i32, i32, vp, i32, i32], sz),
        "oq_route": ([vp, ctypes.c_int, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "oq_route_ws_bytes": ([i64, vp], sz),
        "oq_gemm_w8a8_experts": ([vp, i64, vp, i64, i32, vp, i64, i64, vp, i32, i32, vp, vp, i64, i32, ctypes.c_int, vp, vp, vp,
                                  vp, i64, vp], ctypes.c_int),
        "oq_residual_norm": ([vp, i64, i32, vp, f32, vp, i64, f32, ctypes.c_int, i64, i32, vp, vp, vp, vp, i64, vp, i64, vp],
                             ctypes.c_int),
        "oq_logprobs": ([vp, ctypes.c_int, i64, i64, i32, f32, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "oq_logprobs_ws_bytes": ([i64, i32, i32, i32], sz),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()
EXPORTED = ("oq_last_error", "oq_center", "oq_rotate", "oq_quant_act", "oq_quant_weight",
            "oq_gemm_w4a8", "oq_gemm_w4a4", "oq_linear_fused", "oq_workspace_bytes", "oq_tiled_bytes",
            "oq_prepack_w4", "oq_tiled_mx_bytes", "oq_prepack_mx", "oq_lloyd_max_levels", "oq_lloyd_max_tables",
            "oq_tiled_f16_bytes", "oq_quant_act_lm", "oq_prepack_w16", "oq_gemm_lm", "oq_quant_weight_asym",
            "oq_prepack_w4_asym", "oq_quant_act_gsum", "oq_gemm_w4a4_asym", "oq_kron_plan",
            "oq_linear_fused_noalloc", "oq_probe_mfma", "oq_probe_sink_elems", "oq_quant_weight_w8", "oq_gemm_w8a8",
            "oq_qk_norm_rope", "oq_kv_append", "oq_attn_prefix", "oq_attn_prefix_ws_bytes", "oq_route", "oq_route_ws_bytes",
            "oq_gemm_w8a8_experts", "oq_residual_norm", "oq_logprobs", "oq_logprobs_ws_bytes")


def lib():
    return _lib


def _check(rc: int):
    if rc != OQ_OK:
        raise OQError(rc, _lib.oq_last_error().decode("utf-8", "replace"))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle; the first without the Stream object (2.9 us), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _stream():
    return _raw_stream(torch.cuda.current_device())


def _on(t, dev: int, what: str):
    """t lives on the current device `dev` (get_device() of a host tensor is -1)."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise OQError(OQ_ERR_INVALID_ARG, f"{what} must live on the GPU")
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} lives on GPU {t.get_device()}, the current device is {dev}")


def _current(t: torch.Tensor, what: str):
    """The current device, where `t` has to live, and its current stream."""
    if not t.is_cuda:  # before the runtime is asked
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must live on the GPU")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        _on(t, dev, what)
    return dev, _raw_stream(dev)


_MAX = 0x7FFFFFFF  # the library takes most sizes in 32 bits, and ctypes would pass the remainder of larger ones


def _small(*sizes):
    for n in sizes:
        if not -_MAX <= n <= _MAX:
            raise OQError(OQ_ERR_UNSUPPORTED, f"a size does not fit 32 bits: {sizes}")


def _vec(t: torch.Tensor, n: int, dtype, what: str, dev: int):
    """Address of a contiguous vector of at least n elements of `dtype` on GPU `dev`."""
    if t is None or t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        _need(t, n * dtype.itemsize, what, (dtype,))
        _on(t, dev, what)
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], n: int, dtype, what: str, dev: int):
    return None if t is None else _vec(t, n, dtype, what, dev)


def _dev(t: torch.Tensor):
    if not t.is_cuda:
        raise OQError(OQ_ERR_INVALID_ARG, "tensors must live on the GPU")
    return t.device


def _need(t: Optional[torch.Tensor], nbytes: int, what: str, dtypes=None, optional: bool = False):
    """Argument check before a call: t is a GPU tensor of one of `dtypes`,
    contiguous, holding at least `nbytes` bytes (the library reads or writes
    that many from its base)."""
    if t is None:
        if optional:
            return
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} is required")
    if not t.is_cuda:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must live on the GPU")
    if dtypes is not None and t.dtype not in dtypes:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} holds {t.numel() * t.element_size()} bytes, {nbytes} needed")


_F32 = (torch.float32,)
_BYTES = (torch.uint8, torch.int8)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _out_y(y: Optional[torch.Tensor], M: int, N: int, dev) -> torch.Tensor:
    """The bfloat16 output [M][>= N] (allocated when not given)."""
    if y is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if (not y.is_cuda or y.dtype not in _BF16 or y.dim() != 2 or y.shape[0] < M or y.shape[1] < N
            or y.stride(1) != 1):
        raise OQError(OQ_ERR_INVALID_ARG, f"y must be a GPU bfloat16 matrix of at least {M} x {N} with unit column stride")
    return y


def _epilogue_args(M: int, N: int, mean, w1, bias):
    _need(mean, 4 * M, "mean", _F32, optional=True)
    _need(w1, 4 * N, "w1", _F32, optional=True)
    _need(bias, 4 * N, "bias", _F32, optional=True)


def _bits16(x: torch.Tensor) -> torch.Tensor:
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise OQError(OQ_ERR_INVALID_ARG, "bfloat16 input expected (or its 16-bit pattern)")
    return x


class Rotation:
    """Host descriptor plus the device arrays it points to (kept alive here)."""

    def __init__(self, kind: int, d: int, block: int = 0, rounds: int = 0, perm=None, signs=None, mats=None):
        self.kind, self.d, self.block, self.rounds = kind, d, block, rounds
        self.perm, self.signs, self.mats = perm, signs, mats
        self.c = oq_rot(kind, d, block, rounds, _p(perm), _p(signs), _p(mats))

    @staticmethod
    def rpbh(perm: torch.Tensor, signs: torch.Tensor, block: int) -> "Rotation":
        perm = perm.to(torch.int32).contiguous()
        signs = signs.to(torch.int8).contiguous()
        return Rotation(OQ_ROT_RPBH, perm.shape[-1], block, perm.shape[0], perm=perm, signs=signs)

    @staticmethod
    def kron(n: int) -> "Rotation":
        """The Paley x Sylvester rotation for native width n at the smallest
        admissible padded width (oq_kron_plan)."""
        m, b, npad = oq_kron_plan(n)
        return Rotation(OQ_ROT_KRON, n, b, m)

    @property
    def width(self) -> int:
        """Width of the rotated row (padded for the Kronecker rotation)."""
        return self.rounds * self.block if self.kind == OQ_ROT_KRON else self.d

    @staticmethod
    def dense32(mats_bits: torch.Tensor) -> "Rotation":
        """Per-32-block transforms T_b (bfloat16 bits [d/32][32][32]); the
        weight side uses their inverse-transposes, formed by the library."""
        d = mats_bits.shape[0] * 32
        return Rotation(OQ_ROT_DENSE32, d, 32, 1, mats=mats_bits.contiguous())

    def ref(self):
        return ctypes.byref(self.c)


def _rref(rot: Optional[Rotation]):
    return None if rot is None else rot.ref()


def oq_center(x, xc=None, mean=None):
    x = _bits16(x)
    M, d = x.shape
    dev = _dev(x)
    if mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    ldxc = 0 if xc is None else xc.stride(0)
    _check(_lib.oq_center(_p(x), M, d, x.stride(0), _p(xc), ldxc, _p(mean), _stream()))
    return xc, mean


def oq_rotate(rot: Rotation, x, center: bool = False, y=None, mean=None):
    x = _bits16(x)
    M = x.shape[0]
    dev = _dev(x)
    if y is None:
        y = torch.empty((M, rot.width), dtype=torch.float32, device=dev)
    if center and mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    _check(_lib.oq_rotate(rot.ref(), _p(x), M, x.stride(0), int(center), _p(mean), _p(y), y.stride(0), _stream()))
    return y, mean


def oq_quant_act(x, rot: Optional[Rotation], afmt: int, center: bool = False, codes=None, scale=None,
                 e8m0=None, mean=None):
    x = _bits16(x)
    M, d = x.shape
    dev = _dev(x)
    if rot is not None and rot.kind == OQ_ROT_KRON:
        d = rot.width  # codes have the padded width
    fmt = afmt & ~OQ_SCALE_PCTL  # the scale flag does not change the buffers
    mx_tiled = fmt == (OQ_MXFP4 | OQ_TILED)
    if codes is None and mx_tiled:
        codes = torch.empty(max(16, oq_tiled_mx_bytes(M, d)), dtype=torch.uint8, device=dev)
    elif codes is None and fmt & OQ_TILED:
        planes = 2 if (fmt & ~OQ_TILED) == OQ_A6 else 1
        codes = torch.empty(max(1, planes * oq_tiled_bytes(M, d)), dtype=torch.uint8, device=dev)
    elif codes is None:
        width = d if fmt in (OQ_A8, OQ_A6) else d // 2
        codes = torch.empty((M, width), dtype=torch.int8 if fmt in (OQ_A8, OQ_A6) else torch.uint8, device=dev)
    if mx_tiled:
        if e8m0 is None:
            e8m0 = torch.empty(max(4, oq_tiled_mx_bytes(M, d) // 16), dtype=torch.uint8, device=dev)
    elif fmt == OQ_MXFP4:
        if e8m0 is None:
            e8m0 = torch.empty((M, d // 32), dtype=torch.uint8, device=dev)
    elif scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=dev)
    if center and mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    ldc = 0 if fmt & OQ_TILED else codes.stride(0) * codes.element_size()
    _check(_lib.oq_quant_act(_p(x), M, x.shape[1], x.stride(0), _rref(rot), int(center), afmt, _p(codes),
                             ldc, _p(scale), _p(e8m0), _p(mean), _stream()))
    return {"codes": codes, "scale": scale, "e8m0": e8m0, "mean": mean}


def oq_quant_weight(w, rot: Optional[Rotation], wfmt: int, group: int, codes=None, scales=None, w1=None,
                    want_w1: bool = False):
    N, K = w.shape
    dev = _dev(w)
    Kq = rot.width if rot is not None and rot.kind == OQ_ROT_KRON else K
    if codes is None:
        codes = torch.empty((N, Kq // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = (torch.empty((N, K // 32), dtype=torch.uint8, device=dev) if wfmt == OQ_W_MXFP4
                  else torch.empty((N, Kq // group), dtype=torch.float32, device=dev))
    if want_w1 and w1 is None:
        w1 = torch.empty(N, dtype=torch.float32, device=dev)
    _check(_lib.oq_quant_weight(_p(w), N, K, w.stride(0), _rref(rot), wfmt, group, _p(codes), _p(scales),
                                _p(w1), _stream()))
    return {"codes": codes, "scales": scales, "w1": w1}


def oq_gemm_w4a8(qa, a_scale, w, w_scale, N: int, group: int, mean=None, w1=None, bias=None, y=None,
                 ws=None):
    M, K = qa.shape
    if qa.dtype not in _BYTES or qa.stride(1) != 1:
        raise OQError(OQ_ERR_INVALID_ARG, "qa must be an int8 matrix with unit column stride")
    _need(a_scale, 4 * M, "a_scale", _F32)
    if M and N and group > 0:
        _need(w, N * K // 2, "w", _BYTES)
        _need(w_scale, 4 * N * (K // group), "w_scale", _F32)
    _epilogue_args(M, N, mean, w1, bias)
    _need(ws, 0, "ws", optional=True)
    y = _out_y(y, M, N, _dev(qa))
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.oq_gemm_w4a8(_p(qa), qa.stride(0), _p(a_scale), M, K, _p(w), _p(w_scale), N, group, _p(mean),
                             _p(w1), _p(bias), _p(y), y.stride(0), _p(ws), wsb, _stream()))
    return y


def oq_gemm_w4a4(afmt: int, qa, a_scale, w, w_scale, N: int, group: int, mean=None, w1=None, bias=None,
                 y=None, ws=None, M: Optional[int] = None, K: Optional[int] = None):
    if afmt & OQ_TILED:
        if M is None or K is None:
            raise OQError(OQ_ERR_INVALID_ARG, "tiled operands need explicit M and K")
        lda = 0
        if M > 0 and N > 0 and K > 0:
            if afmt == (OQ_MXFP4 | OQ_TILED):
                _need(qa, oq_tiled_mx_bytes(M, K), "qa", _BYTES)
                _need(a_scale, oq_tiled_mx_bytes(M, K) // 16, "a_scale", _BYTES)
                _need(w, oq_tiled_mx_bytes(N, K), "w", _BYTES)
                _need(w_scale, oq_tiled_mx_bytes(N, K) // 16, "w_scale", _BYTES)
            else:
                planes = 2 if (afmt & ~OQ_TILED) == OQ_A6 else 1
                _need(qa, planes * oq_tiled_bytes(M, K), "qa", _BYTES)
                _need(a_scale, 4 * M, "a_scale", _F32)
                _need(w, oq_tiled_bytes(N, K), "w", _BYTES)
                _need(w_scale, 4 * (K // 64) * ((N + 31) // 32 * 32), "w_scale", _F32)
    else:
        M = qa.shape[0]
        K = qa.shape[1] * 2
        lda = qa.stride(0) * qa.element_size()
        if qa.dtype not in _BYTES or qa.stride(1) != 1:
            raise OQError(OQ_ERR_INVALID_ARG, "qa must be a uint8 matrix with unit column stride")
        if M > 0 and N > 0:
            _need(w, N * K // 2, "w", _BYTES)
            if afmt == OQ_MXFP4:
                _need(a_scale, M * (K // 32), "a_scale", _BYTES)
                _need(w_scale, N * (K // 32), "w_scale", _BYTES)
            elif group > 0:
                _need(a_scale, 4 * M, "a_scale", _F32)
                _need(w_scale, 4 * N * (K // group), "w_scale", _F32)
    _epilogue_args(M, N, mean, w1, bias)
    y = _out_y(y, M, N, _dev(qa))
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.oq_gemm_w4a4(afmt, _p(qa), lda, _p(a_scale), M, K, _p(w),
                             _p(w_scale), N, group, _p(mean), _p(w1), _p(bias), _p(y), y.stride(0), _p(ws), wsb,
                             _stream()))
    return y


def oq_tiled_bytes(rows: int, K: int) -> int:
    return int(_lib.oq_tiled_bytes(rows, K))


def oq_prepack_w4(w, w_scale, N: int, K: int, group: int = 64, w_tiled=None, w_scale_t=None):
    dev = _dev(w)
    if w_tiled is None:
        w_tiled = torch.empty(max(1, oq_tiled_bytes(N, K)), dtype=torch.uint8, device=dev)
    if w_scale_t is None:
        w_scale_t = torch.empty((K // 64, (N + 31) // 32 * 32), dtype=torch.float32, device=dev)
    _check(_lib.oq_prepack_w4(_p(w), _p(w_scale), N, K, group, _p(w_tiled), _p(w_scale_t), _stream()))
    return {"codes": w_tiled, "scales": w_scale_t}


def oq_tiled_mx_bytes(rows: int, K: int) -> int:
    return int(_lib.oq_tiled_mx_bytes(rows, K))


def oq_prepack_mx(w, w_e8m0, N: int, K: int, w_tiled=None, w_e8m0_tiled=None):
    dev = _dev(w)
    nb = oq_tiled_mx_bytes(N, K)
    if w_tiled is None:
        w_tiled = torch.empty(max(16, nb), dtype=torch.uint8, device=dev)
    if w_e8m0_tiled is None:
        w_e8m0_tiled = torch.empty(max(4, nb // 16), dtype=torch.uint8, device=dev)
    _check(_lib.oq_prepack_mx(_p(w), _p(w_e8m0), N, K, _p(w_tiled), _p(w_e8m0_tiled), _stream()))
    return {"codes": w_tiled, "scales": w_e8m0_tiled}


def oq_workspace_bytes(op: int, M: int, K: int, N: int, afmt: int) -> int:
    return int(_lib.oq_workspace_bytes(op, M, K, N, afmt))


def oq_linear_fused(x, rot: Optional[Rotation], center: bool, afmt: int, w, w_scale, N: int, group: int,
                    w1=None, bias=None, y=None, ws=None):
    x = _bits16(x)
    M, K = x.shape
    dev = _dev(x)
    fmt = afmt & ~OQ_SCALE_PCTL
    if M > 0 and N > 0:
        if fmt == (OQ_MXFP4 | OQ_TILED):
            _need(w, oq_tiled_mx_bytes(N, K), "w", _BYTES)
            _need(w_scale, oq_tiled_mx_bytes(N, K) // 16, "w_scale", _BYTES)
        elif fmt & OQ_TILED:
            _need(w, oq_tiled_bytes(N, K), "w", _BYTES)
            _need(w_scale, 4 * (K // 64) * ((N + 31) // 32 * 32), "w_scale", _F32)
        else:
            _need(w, N * K // 2, "w", _BYTES)
            if fmt == OQ_MXFP4:
                _need(w_scale, N * (K // 32), "w_scale", _BYTES)
            elif group > 0:
                _need(w_scale, 4 * N * (K // group), "w_scale", _F32)
    _epilogue_args(M, N, None, w1, bias)
    y = _out_y(y, M, N, dev)
    if ws is None:
        ws = torch.empty(max(1, oq_workspace_bytes(OQ_OP_LINEAR, M, K, N, afmt)), dtype=torch.uint8, device=dev)
    _check(_lib.oq_linear_fused(_p(x), M, K, x.stride(0), _rref(rot), int(center), afmt, _p(w), _p(w_scale), N,
                                group, _p(w1), _p(bias), _p(y), y.stride(0), _p(ws), ws.numel(), _stream()))
    return y


OQ_PROBE_FP6, OQ_PROBE_FP4, OQ_PROBE_FP8, OQ_PROBE_I8, OQ_PROBE_BF16, OQ_PROBE_F16 = 1, 2, 3, 4, 5, 6
OQ_PROBE_FP6_UPDATE = 7


def oq_probe_mfma(kind: int, iters: int, sink=None):
    """Launches the matrix-core rate probe on the current stream; returns
    (operation count of the launch, sink).  The caller times it."""
    if sink is None:
        sink = torch.empty(int(_lib.oq_probe_sink_elems()), dtype=torch.float32, device="cuda")
    _need(sink, 4 * int(_lib.oq_probe_sink_elems()), "sink", _F32)
    ops = ctypes.c_double(0.0)
    _check(_lib.oq_probe_mfma(kind, iters, _p(sink), ctypes.byref(ops), _stream()))
    return ops.value, sink


OQ_NOALLOC_SCRATCH_BYTES = 32 << 20


def oq_linear_fused_noalloc(x, rot: Optional[Rotation], center: bool, afmt: int, w, w_scale, N: int, group: int,
                            w1=None, bias=None, y=None):
    """oq_linear_fused without a workspace: the library's static per-GPU
    scratch holds the codes (calls on one GPU must not overlap)."""
    x = _bits16(x)
    M, K = x.shape
    dev = _dev(x)
    _epilogue_args(M, N, None, w1, bias)
    y = _out_y(y, M, N, dev)
    _check(_lib.oq_linear_fused_noalloc(_p(x), M, K, x.stride(0), _rref(rot), int(center), afmt, _p(w), _p(w_scale),
                                        N, group, _p(w1), _p(bias), _p(y), y.stride(0), _stream()))
    return y


# ---------------------------------------------------------------- Lloyd-Max path
def oq_lloyd_max_levels(d: int, bits: int) -> np.ndarray:
    """Host call: float64 levels [2^bits] of the Lloyd-Max codebook for width d."""
    out = np.zeros(1 << bits, dtype=np.float64)
    _check(_lib.oq_lloyd_max_levels(d, bits, out.ctypes.data_as(ctypes.c_void_p)))
    return out


def oq_lloyd_max_tables(d: int, bits: int):
    """Host call: (float16 level bits uint16 [2^bits], float32 thresholds [2^bits - 1])."""
    lv = np.zeros(1 << bits, dtype=np.uint16)
    thr = np.zeros((1 << bits) - 1, dtype=np.float32)
    _check(_lib.oq_lloyd_max_tables(d, bits, lv.ctypes.data_as(ctypes.c_void_p),
                                    thr.ctypes.data_as(ctypes.c_void_p)))
    return lv, thr


def oq_tiled_f16_bytes(rows: int, K: int) -> int:
    return int(_lib.oq_tiled_f16_bytes(rows, K))


def oq_quant_act_lm(x, rot: Optional[Rotation], bits: int, levels, thresholds, tiled: bool = False,
                    center: bool = False, codes=None, scale=None, mean=None):
    """levels: device uint16/int16 float16 bits [2^bits]; thresholds: device float32."""
    x = _bits16(x)
    M, d = x.shape
    dev = _dev(x)
    if codes is None and tiled:
        codes = torch.empty(max(16, oq_tiled_f16_bytes(M, d)), dtype=torch.uint8, device=dev)
    elif codes is None:
        codes = torch.empty((M, d // 2 if bits <= 4 else d), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=dev)
    if center and mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    ldc = 0 if tiled else codes.stride(0) * codes.element_size()
    _check(_lib.oq_quant_act_lm(_p(x), M, d, x.stride(0), _rref(rot), int(center), bits, int(tiled), _p(levels),
                                _p(thresholds), _p(codes), ldc, _p(scale), _p(mean), _stream()))
    return {"codes": codes, "scale": scale, "mean": mean}


def oq_prepack_w16(w, w_scale, N: int, K: int, group: int, w16=None):
    dev = _dev(w)
    if w16 is None:
        w16 = torch.empty(max(16, oq_tiled_f16_bytes(N, K)) // 2, dtype=torch.int16, device=dev)
    _check(_lib.oq_prepack_w16(_p(w), _p(w_scale), N, K, group, _p(w16), _stream()))
    return w16


def oq_gemm_lm(bits: int, qa, a_scale, w16, N: int, levels=None, tiled: bool = False, mean=None, w1=None,
               bias=None, y=None, ws=None, M: Optional[int] = None, K: Optional[int] = None):
    if tiled:
        if M is None or K is None:
            raise OQError(OQ_ERR_INVALID_ARG, "tiled operands need explicit M and K")
        lda = 0
        if M > 0 and N > 0 and K > 0:
            _need(qa, oq_tiled_f16_bytes(M, K), "qa")
    else:
        M = qa.shape[0]
        K = qa.shape[1] * (2 if bits <= 4 else 1)
        lda = qa.stride(0) * qa.element_size()
        if ws is None:
            ws = torch.empty(max(16, oq_workspace_bytes(OQ_OP_GEMM_LM, M, K, N, 0)), dtype=torch.uint8,
                             device=_dev(qa))
    if M > 0 and N > 0 and K > 0:
        _need(a_scale, 4 * M, "a_scale", _F32)
        _need(w16, oq_tiled_f16_bytes(N, K), "w16")
    _epilogue_args(M, N, mean, w1, bias)
    y = _out_y(y, M, N, _dev(qa))
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.oq_gemm_lm(bits, int(tiled), _p(qa), lda, _p(a_scale), M, K, _p(levels), _p(w16), N, _p(mean),
                           _p(w1), _p(bias), _p(y), y.stride(0), _p(ws), wsb, _stream()))
    return y


# ---------------------------------------------------------------- asymmetric weights
def oq_quant_weight_asym(w, rot: Optional[Rotation], group: int, codes=None, sigma=None, zero=None, w1=None,
                         want_w1: bool = False):
    N, K = w.shape
    dev = _dev(w)
    Kq = rot.width if rot is not None and rot.kind == OQ_ROT_KRON else K
    if codes is None:
        codes = torch.empty((N, Kq // 2), dtype=torch.uint8, device=dev)
    if sigma is None:
        sigma = torch.empty((N, Kq // group), dtype=torch.int16, device=dev)
    if zero is None:
        zero = torch.empty((N, Kq // group), dtype=torch.int16, device=dev)
    if want_w1 and w1 is None:
        w1 = torch.empty(N, dtype=torch.float32, device=dev)
    _check(_lib.oq_quant_weight_asym(_p(w), N, K, w.stride(0), _rref(rot), group, _p(codes), _p(sigma), _p(zero),
                                     _p(w1), _stream()))
    return {"codes": codes, "sigma": sigma, "zero": zero, "w1": w1}


def oq_prepack_w4_asym(w, sigma, zero, N: int, K: int, group: int = 64):
    dev = _dev(w)
    Np = (N + 31) // 32 * 32
    w_tiled = torch.empty(max(16, oq_tiled_bytes(N, K)), dtype=torch.uint8, device=dev)
    w_scale_t = torch.empty((K // 64, Np), dtype=torch.float32, device=dev)
    corr = torch.empty((K // 64, Np, 2), dtype=torch.int32, device=dev)
    _check(_lib.oq_prepack_w4_asym(_p(w), _p(sigma), _p(zero), N, K, group, _p(w_tiled), _p(w_scale_t), _p(corr),
                                   _stream()))
    return {"codes": w_tiled, "scales": w_scale_t, "corr": corr}


def oq_quant_act_gsum(x, rot: Optional[Rotation], afmt: int, center: bool = False, codes=None, scale=None,
                      gsum=None, mean=None):
    x = _bits16(x)
    M, d = x.shape
    dev = _dev(x)
    fmt = afmt & ~OQ_SCALE_PCTL
    if codes is None:
        planes = 2 if (fmt & ~OQ_TILED) == OQ_A6 else 1
        codes = torch.empty(max(16, planes * oq_tiled_bytes(M, d)), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=dev)
    if gsum is None:  # one word per (group, row): two bfloat16 pieces of the group sum
        gsum = torch.empty((d // 64, M), dtype=torch.int32, device=dev)
    if center and mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    _check(_lib.oq_quant_act_gsum(_p(x), M, d, x.stride(0), _rref(rot), int(center), afmt, _p(codes), _p(scale),
                                  _p(gsum), _p(mean), _stream()))
    return {"codes": codes, "scale": scale, "gsum": gsum, "mean": mean}


def oq_gemm_w4a4_asym(qa, a_scale, gsum, w, N: int, M: int, K: int, mean=None, w1=None, bias=None, y=None,
                      afmt: int = OQ_A4 | OQ_TILED):
    """w: oq_prepack_w4_asym output (dict with codes, scales, corr)."""
    if M > 0 and N > 0 and K > 0:
        Np = (N + 31) // 32 * 32
        _need(qa, oq_tiled_bytes(M, K), "qa", _BYTES)
        _need(a_scale, 4 * M, "a_scale", _F32)
        _need(gsum, 4 * (K // 64) * M, "gsum")
        _need(w["codes"], oq_tiled_bytes(N, K), "w codes", _BYTES)
        _need(w["scales"], 4 * (K // 64) * Np, "w scales", _F32)
        _need(w["corr"], 8 * (K // 64) * Np, "w corr")
    _epilogue_args(M, N, mean, w1, bias)
    y = _out_y(y, M, N, _dev(qa))
    _check(_lib.oq_gemm_w4a4_asym(afmt, _p(qa), _p(a_scale), _p(gsum), M, K, _p(w["codes"]), _p(w["scales"]),
                                  _p(w["corr"]), N, _p(mean), _p(w1), _p(bias), _p(y), y.stride(0), _stream()))
    return y


def oq_kron_plan(n: int):
    """Host call: (m, block, n_pad), the smallest admissible padded width."""
    m, b, p = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.oq_kron_plan(n, ctypes.byref(m), ctypes.byref(b), ctypes.byref(p)))
    return m.value, b.value, p.value


# ---------------------------------------------------------------- 8-bit weights
def oq_quant_weight_w8(w, rot: Optional[Rotation] = None, codes=None, scales=None, w1=None, want_w1: bool = False):
    if w.dim() != 2 or w.dtype != torch.float32 or w.stride(1) != 1:
        raise OQError(OQ_ERR_INVALID_ARG, "w must be a float32 matrix with unit column stride")
    N, K = w.shape
    _small(N, K)
    on, stream = _current(w, "w")
    dev = w.device
    for t in () if rot is None else (rot.perm, rot.signs, rot.mats):
        if t is not None:
            _on(t, on, "the rotation")
    Kq = rot.width if rot is not None else K
    if codes is None:
        codes = torch.empty((N, Kq), dtype=torch.int8, device=dev)
    elif not codes.is_cuda or codes.dtype != torch.int8 or codes.dim() != 2 or codes.shape[0] < N \
            or codes.shape[1] < Kq or codes.stride(1) != 1:
        raise OQError(OQ_ERR_INVALID_ARG, f"codes must be a GPU int8 matrix of at least {N} x {Kq}")
    if scales is None:
        scales = torch.empty(N, dtype=torch.float32, device=dev)
    if want_w1 and w1 is None:
        w1 = torch.empty(N, dtype=torch.float32, device=dev)
    _on(codes, on, "codes")
    _check(_lib.oq_quant_weight_w8(_p(w), N, K, w.stride(0), _rref(rot), _p(codes), codes.stride(0),
                                   _vec(scales, N, _F, "scales", on), _opt(w1, N, _F, "w1", on), stream))
    return {"codes": codes, "scales": scales, "w1": w1}


def oq_gemm_w8a8(qa, a_scale, w, w_scale, mean=None, w1=None, bias=None, y=None):
    """qa int8 [M][K] (oq_quant_act OQ_A8 or OQ_A6 codes), w int8 [N][K] (oq_quant_weight_w8)."""
    if qa.dim() != 2 or w.dim() != 2 or qa.dtype != torch.int8 or w.dtype != torch.int8:
        raise OQError(OQ_ERR_INVALID_ARG, "qa and w must be int8 matrices")
    (M, K), (N, Kw) = qa.shape, w.shape
    (lda, ca), (ldw, cw) = qa.stride(), w.stride()
    if K != Kw or ca != 1 or cw != 1:
        raise OQError(OQ_ERR_INVALID_ARG, f"qa [M][K] and w [N][K] with unit column strides, got {qa.shape} and {w.shape}")
    if K > _MAX or N > _MAX:
        _small(K, N)
    dev, stream = _current(qa, "qa")
    if w.get_device() != dev:
        _on(w, dev, "w")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    elif y.dtype not in _BF16 or y.dim() != 2 or y.shape[0] < M or y.shape[1] < N:
        _out_y(y, M, N, qa.device)
    ldy, cy = y.stride()
    if cy != 1:
        _out_y(y, M, N, qa.device)
    if y.get_device() != dev:
        _on(y, dev, "y")
    # a matrix of one row has no row stride to speak of
    _check(_lib.oq_gemm_w8a8(qa.data_ptr(), lda if M > 1 else (K + 15) // 16 * 16, _vec(a_scale, M, _F, "a_scale", dev), M, K,
                             w.data_ptr(), ldw if N > 1 else (K + 15) // 16 * 16, _vec(w_scale, N, _F, "w_scale", dev), N,
                             _opt(mean, M, _F, "mean", dev), _opt(w1, N, _F, "w1", dev), _opt(bias, N, _F, "bias", dev),
                             y.data_ptr(), ldy if M > 1 else N, stream))
    return y


# ---------------------------------------------------------------- heads, cache, attention
class oq_rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int64), ("dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class oq_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("pages", ctypes.c_int32),
                ("page", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32)]


class Rope:
    """Rotary tables cos, sin (float32 [rows][dim / 2], kept alive here) and the order of the pairs."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool = False):
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise OQError(OQ_ERR_INVALID_ARG, "cos and sin must be matrices of one shape")
        for t, what in ((cos, "cos"), (sin, "sin")):
            _need(t, 0, what, _F32)
        _small(2 * cos.shape[1])
        self.dev = cos.get_device()
        _on(sin, self.dev, "sin")
        self.cos, self.sin, self.interleaved = cos, sin, interleaved
        self.c = oq_rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(interleaved))
        self.ref = ctypes.byref(self.c)


class PagedKV:
    """A paged cache: k and v bfloat16 [pages][heads][page][d] (kept alive
    here), contiguous but for one stride from page to page shared by both."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t, what in ((k, "k"), (v, "v")):
            if not t.is_cuda or t.dtype not in _BF16 or t.dim() != 4:
                raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be a GPU bfloat16 tensor [pages][heads][page][d]")
            if t.stride()[1:] != (t.shape[2] * t.shape[3], t.shape[3], 1):
                raise OQError(OQ_ERR_INVALID_ARG, f"the pages of {what} must be contiguous")
        self.dev = k.get_device()
        if k.shape != v.shape or k.stride() != v.stride() or v.get_device() != self.dev:
            raise OQError(OQ_ERR_INVALID_ARG, "k and v must have one shape, stride and device")
        self.k, self.v = k, v
        _small(*k.shape)
        self.pages, self.heads, self.page, self.d = k.shape
        self.c = oq_kv(k.data_ptr(), v.data_ptr(), k.stride(0), self.pages, self.page, self.heads, self.d)
        self.ref = ctypes.byref(self.c)


def _handle(h, dev: int, what: str):
    """Reference to the descriptor of a Rope or PagedKV, whose tensors have to live on GPU `dev`."""
    if h.dev != dev:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} lives on GPU {h.dev}, the current device is {dev}")
    return h.ref


def _heads(t: torch.Tensor, shape, what: str, dev: int):
    """(address, token stride, head stride) of a bfloat16 tensor [T][heads][d] on GPU `dev`."""
    if t.get_device() != dev:
        _on(t, dev, what)
    if t.shape != shape or t.dtype not in _BF16:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be a GPU bfloat16 tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    ld, hs, es = t.stride()
    if es != 1:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must have unit stride within a head")
    return t.data_ptr(), ld, hs


def _tokens(t: torch.Tensor, what: str):
    if t.dim() != 3:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be a tensor [T][heads][d]")
    return t.shape


_F, _I32, _I64 = torch.float32, torch.int32, torch.int64


def oq_qk_norm_rope(q, k, w_q=None, w_k=None, eps: float = 1e-6, rope: Optional[Rope] = None, pos=None, q_out=None,
                    k_out=None):
    """q [T][heads_q][d], k [T][heads_k][d] (either may be None), any token and
    head strides; returns (q_out, k_out).  Passing q as q_out works in place."""
    x = q if q is not None else k
    if x is None:
        raise OQError(OQ_ERR_INVALID_ARG, "q or k is required")
    T, heads, d = _tokens(x, "q" if q is not None else "k")
    if heads > _MAX or d > _MAX or (k is not None and _tokens(k, "k")[1] > _MAX):
        raise OQError(OQ_ERR_UNSUPPORTED, "head counts and widths past 32 bits")
    dev, stream = _current(x, "q" if q is not None else "k")
    args = [None, 0, 0, 0, None, 0, 0, 0]
    outs = [None, 0, 0, None, 0, 0]
    if q is not None:
        shape = q.shape
        q_out = torch.empty(shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        args[0:4] = *_heads(q, shape, "q", dev), shape[1]
        outs[0:3] = _heads(q_out, shape, "q_out", dev)
    if k is not None:
        shape = k.shape
        if shape[0] != T or shape[2] != d:
            raise OQError(OQ_ERR_INVALID_ARG, f"q and k differ: {tuple(x.shape)}, {tuple(shape)}")
        k_out = torch.empty(shape, dtype=k.dtype, device=k.device) if k_out is None else k_out
        args[4:8] = *_heads(k, shape, "k", dev), shape[1]
        outs[3:6] = _heads(k_out, shape, "k_out", dev)
    _check(_lib.oq_qk_norm_rope(*args, T, d, _opt(w_q, d, _F, "w_q", dev), _opt(w_k, d, _F, "w_k", dev), eps,
                                None if rope is None else _handle(rope, dev, "rope"), _opt(pos, T, _I32, "pos", dev), *outs,
                                stream))
    return q_out, k_out


def oq_kv_append(k, v, slot, kv: PagedKV, w_k=None, eps: float = 1e-6, rope: Optional[Rope] = None, pos=None):
    """k, v [T][heads][d] into the places slot (int64 [T], negative: skipped) of the cache."""
    T, d = k.shape[0], kv.d
    dev, stream = _current(k, "k")
    shape = (T, kv.heads, d)
    _check(_lib.oq_kv_append(*_heads(k, shape, "k", dev), *_heads(v, shape, "v", dev), T, _opt(w_k, d, _F, "w_k", dev), eps,
                             None if rope is None else _handle(rope, dev, "rope"), _opt(pos, T, _I32, "pos", dev),
                             _vec(slot, T, _I64, "slot", dev), _handle(kv, dev, "kv"), stream))


def oq_attn_prefix_ws_bytes(B: int, n_q: int, heads_q: int, kv: PagedKV, prefix_len: int, table_ld: int) -> int:
    """Scratch bytes of one call; a shorter prefix can take more than a longer one."""
    _small(B, n_q, heads_q, prefix_len, table_ld)
    return int(_lib.oq_attn_prefix_ws_bytes(B, n_q, heads_q, kv.ref, prefix_len, table_ld))


def oq_attn_prefix(q, n_q: int, kv: PagedKV, prefix_table, prefix_len: int, tables, lens, scale: float, o=None, lse=None,
                   ws=None, want_lse: bool = False):
    """q [B n_q][heads_q][d]; prefix_table int32 [>= ceil(prefix_len / page)] (None
    without a prefix); tables int32 [B][table_ld] and lens int32 [B] (both None
    without suffixes); returns (o, lse)."""
    shape = _tokens(q, "q")
    T, heads_q, d = shape
    if n_q < 1 or T % n_q or d != kv.d:
        raise OQError(OQ_ERR_INVALID_ARG, f"q of shape {tuple(shape)} for n_q={n_q} and heads of {kv.d}")
    B = T // n_q
    if T > _MAX or heads_q > _MAX or prefix_len > _MAX:
        _small(B, n_q, heads_q, prefix_len)
    dev, stream = _current(q, "q")
    table_ld, table_at, lens_at = 0, None, None
    if tables is not None:
        if tables.dim() != 2 or tables.shape[0] != B:
            raise OQError(OQ_ERR_INVALID_ARG, f"tables must be a matrix of {B} rows")
        table_ld = tables.shape[1]
        if table_ld > _MAX:
            _small(table_ld)
        table_at, lens_at = _vec(tables, 0, _I32, "tables", dev), _vec(lens, B, _I32, "lens", dev)
    if o is None:
        o = torch.empty(shape, dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, heads_q), dtype=_F, device=q.device)
    if ws is None:
        ws = torch.empty(oq_attn_prefix_ws_bytes(B, n_q, heads_q, kv, prefix_len, table_ld), dtype=torch.uint8, device=q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise OQError(OQ_ERR_INVALID_ARG, f"ws must be a contiguous tensor on GPU {dev}")
    prefix_at = _vec(prefix_table, -(-prefix_len // kv.page), _I32, "prefix_table", dev) if prefix_len > 0 else None
    _check(_lib.oq_attn_prefix(*_heads(q, shape, "q", dev), B, n_q, heads_q, _handle(kv, dev, "kv"), prefix_at, prefix_len,
                               table_at, table_ld, lens_at, scale, *_heads(o, shape, "o", dev),
                               _opt(lse, T * heads_q, _F, "lse", dev), ws.data_ptr(), ws.numel() * ws.element_size(), stream))
    return o, lse


# ---------------------------------------------------------------- sparse layers, residual stream, answers
class oq_router(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("experts", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_best", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("factor", ctypes.c_float)]


class oq_norm(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("b", ctypes.c_void_p), ("kind", ctypes.c_int32), ("eps", ctypes.c_float)]


class oq_mod(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p), ("row", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("rows", ctypes.c_int64)]


_SCORES = {"softmax": OQ_SCORE_SOFTMAX, "sigmoid": OQ_SCORE_SIGMOID}


class Router:
    """How tokens choose k of `experts`: scores ("softmax" or "sigmoid"), a balance
    bias (float32 [experts], kept alive here), groups of which the best top_groups are
    open (by the sum of their group_best best), weights renormalised over the chosen
    or not, and a factor on them."""

    def __init__(self, experts: int, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
                 top_groups: Optional[int] = None, group_best: int = 1, renorm: bool = True, factor: float = 1.0):
        if score not in _SCORES:
            raise OQError(OQ_ERR_INVALID_ARG, f"score must be one of {tuple(_SCORES)}, got {score!r}")
        top_groups = groups if top_groups is None else top_groups
        _small(experts, k, groups, top_groups, group_best)
        self.dev = None
        if bias is not None:
            _need(bias, 4 * experts, "bias", _F32)
            self.dev = bias.get_device()
        self.experts, self.k, self.bias = experts, k, bias
        self.c = oq_router(None if bias is None else bias.data_ptr(), experts, k, _SCORES[score], groups, top_groups, group_best,
                           int(renorm), factor)
        self.ref = ctypes.byref(self.c)


class Norm:
    """An RMS or layer norm (OQ_NORM_RMS, OQ_NORM_LAYER) of rows of d with weights
    and bias (float32 [d], kept alive here; each may be None)."""

    def __init__(self, kind: int, d: int, eps: float = 1e-6, w: Optional[torch.Tensor] = None, b: Optional[torch.Tensor] = None):
        self.dev = None
        for t, what in ((w, "w"), (b, "b")):
            if t is None:
                continue
            _need(t, 4 * d, what, _F32)
            if self.dev is not None:
                _on(t, self.dev, what)
            self.dev = t.get_device()
        self.d, self.w, self.b = d, w, b
        self.c = oq_norm(None if w is None else w.data_ptr(), None if b is None else b.data_ptr(), kind, eps)
        self.ref = ctypes.byref(self.c)


def _wide(h, dev: int, what: str):
    """Reference to a Router's or Norm's descriptor, whose tensors (if any) have to live on GPU `dev`."""
    if h.dev is not None and h.dev != dev:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} lives on GPU {h.dev}, the current device is {dev}")
    return h.ref


_TYPES = {torch.float32: OQ_F32, torch.bfloat16: OQ_BF16}


def _matrix(t: torch.Tensor, shape, dtypes, what: str, dev: int):
    """(address, row stride) of a matrix of `shape` with unit column stride on GPU `dev`."""
    if t.get_device() != dev:
        _on(t, dev, what)
    if t.dim() != 2 or tuple(t.shape) != tuple(shape) or t.dtype not in dtypes or (t.stride(1) != 1 and shape[1] > 1):
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be a matrix of shape {tuple(shape)} and type {dtypes} with unit column stride, "
                      f"got {t.dtype} {tuple(t.shape)}, strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]  # a matrix of one row has no row stride to speak of


def _logits(t: torch.Tensor, what: str):
    """(type, address, row stride) of logits [T][V] on the current device."""
    dev, stream = _current(t, what)
    if t.dim() != 2 or t.dtype not in _TYPES:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} must be a float32 or bfloat16 matrix, got {t.dtype} {tuple(t.shape)}")
    return dev, stream, _TYPES[t.dtype], *_matrix(t, t.shape, _TYPES, what, dev)


def _scratch(ws, nbytes, dev: int, device):
    """(tensor, address, bytes) of a workspace; where none is given, one of nbytes() is allocated."""
    if ws is None:
        ws = torch.empty(nbytes(), dtype=torch.uint8, device=device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise OQError(OQ_ERR_INVALID_ARG, f"ws must be a contiguous tensor on GPU {dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def oq_route_ws_bytes(T: int, router: Router) -> int:
    """Scratch bytes of one call with lists."""
    return int(_lib.oq_route_ws_bytes(T, router.ref))


def oq_route(logits, router: Router, mask=None, ids=None, weights=None, offsets=None, order=None, ws=None, lists: bool = True):
    """logits float32 or bfloat16 [T][experts]; mask uint8 or bool [T] (0: a token
    without experts); returns (ids int32 [T][k], weights float32 [T][k], offsets int32
    [experts + 1], order int32 [T k]), the last two None without lists."""
    dev, stream, dtype, at, ld = _logits(logits, "logits")
    T, E, k = logits.shape[0], router.experts, router.k
    if logits.shape[1] != E:
        raise OQError(OQ_ERR_INVALID_ARG, f"logits of {logits.shape[1]} columns for {E} experts")
    if ids is None:
        ids = torch.empty((T, k), dtype=_I32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, k), dtype=_F, device=logits.device)
    if lists:
        if offsets is None:
            offsets = torch.empty(E + 1, dtype=_I32, device=logits.device)
        if order is None:
            order = torch.empty(T * k, dtype=_I32, device=logits.device)
    elif offsets is not None or order is not None:
        raise OQError(OQ_ERR_INVALID_ARG, "offsets or order with lists=False")
    ws, ws_at, ws_bytes = _scratch(ws, lambda: oq_route_ws_bytes(T, router) if lists else 0, dev, logits.device)
    mask_at = None
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool):
            raise OQError(OQ_ERR_INVALID_ARG, f"mask must be uint8 or bool, got {mask.dtype}")
        mask_at = _vec(mask, T, mask.dtype, "mask", dev)
    _check(_lib.oq_route(at, dtype, ld, T, mask_at, _wide(router, dev, "the router"), _vec(ids, T * k, _I32, "ids", dev),
                         _vec(weights, T * k, _F, "weights", dev), _opt(offsets, E + 1, _I32, "offsets", dev),
                         _opt(order, T * k, _I32, "order", dev), ws_at, ws_bytes, stream))
    return ids, weights, offsets, order


def oq_gemm_w8a8_experts(qa, a_scale, w, w_scale, offsets, order, per: int = 1, act: int = OQ_ACT_NONE, mean=None, w1=None,
                         bias=None, y=None):
    """qa int8 [rows][K], a_scale and mean float32 [rows]; w int8 [E][N][K], w_scale,
    w1 and bias float32 [E][N]; offsets int32 [E + 1] and order int32 [n] from
    oq_route; entry i uses activation row i / per and writes row i of y bfloat16 [n][N]
    ([n][N / 2] with OQ_ACT_SWIGLU)."""
    if qa.dim() != 2 or w.dim() != 3 or qa.dtype != torch.int8 or w.dtype != torch.int8:
        raise OQError(OQ_ERR_INVALID_ARG, "qa must be an int8 matrix and w an int8 tensor [E][N][K]")
    (rows, K), (E, N, Kw) = qa.shape, w.shape
    if K != Kw or qa.stride(1) != 1 or w.stride(2) != 1:
        raise OQError(OQ_ERR_INVALID_ARG, f"qa [rows][K] and w [E][N][K] with unit column strides, got {tuple(qa.shape)} and {tuple(w.shape)}")
    _small(K, N, E, per)
    dev, stream = _current(qa, "qa")
    _on(w, dev, "w")
    n = order.numel()
    out = N // 2 if act == OQ_ACT_SWIGLU else N
    if y is None:
        y = torch.empty((n, out), dtype=torch.bfloat16, device=qa.device)
    y_at, ldy = _matrix(y, (n, out), _BF16, "y", dev)
    pad = (K + 15) // 16 * 16
    ldw = w.stride(1) if N > 1 else pad
    _check(_lib.oq_gemm_w8a8_experts(qa.data_ptr(), qa.stride(0) if rows > 1 else pad, _vec(a_scale, rows, _F, "a_scale", dev), rows, K,
                                     w.data_ptr(), ldw, w.stride(0) if E > 1 else N * ldw, _vec(w_scale, E * N, _F, "w_scale", dev),
                                     N, E, _vec(offsets, E + 1, _I32, "offsets", dev), _vec(order, n, _I32, "order", dev), n, per, act,
                                     _opt(mean, rows, _F, "mean", dev), _opt(w1, E * N, _F, "w1", dev),
                                     _opt(bias, E * N, _F, "bias", dev), y_at, ldy, stream))
    return y


def oq_residual_norm(y, r=None, weights=None, post: Optional[Norm] = None, pre: Optional[Norm] = None, gate=None, scale=None,
                     shift=None, row=None, y_scale: float = 1.0, r_scale: float = 1.0, r_out=None, h=None, want_r: bool = True,
                     want_h: bool = True, r_dtype=torch.bfloat16):
    """y bfloat16 [T k][d] (None: no block output) with weights float32 [T][k] (None:
    k = 1); r float32 or bfloat16 [T][d] (None: no residual yet, r_out is of r_dtype);
    gate, scale, shift bfloat16 [rows][d] of one row stride, row int32 [T]; returns
    (r_out, h), None where not wanted.  Passing r as r_out works in place."""
    x = y if y is not None else r
    if x is None or x.dim() != 2:
        raise OQError(OQ_ERR_INVALID_ARG, "y or r, a matrix, is required")
    d = x.shape[1]
    dev, stream = _current(x, "y" if y is not None else "r")
    k = 1
    if weights is not None:
        if weights.dim() != 2 or y is None or weights.shape[0] * weights.shape[1] != y.shape[0]:
            raise OQError(OQ_ERR_INVALID_ARG, "weights must be a matrix of as many elements as y has rows")
        k = weights.shape[1]
        T = weights.shape[0]
    else:
        T = x.shape[0]
    _small(d, k)
    r_type = r.dtype if r is not None else r_out.dtype if r_out is not None else r_dtype
    if r_type not in _TYPES:
        raise OQError(OQ_ERR_INVALID_ARG, f"r and r_out must be float32 or bfloat16, got {r_type}")
    if want_r and r_out is None:
        r_out = torch.empty((T, d), dtype=r_type, device=x.device)
    if want_h and h is None:
        h = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
    none = (None, 0)
    y_at, y_ld = none if y is None else _matrix(y, (T * k, d), _BF16, "y", dev)
    r_at, r_ld = none if r is None else _matrix(r, (T, d), (r_type,), "r", dev)
    ro_at, ro_ld = none if not want_r else _matrix(r_out, (T, d), (r_type,), "r_out", dev)
    h_at, h_ld = none if not want_h else _matrix(h, (T, d), _BF16, "h", dev)
    for n, what in ((post, "post"), (pre, "pre")):
        if n is not None and n.d != d:
            raise OQError(OQ_ERR_INVALID_ARG, f"{what} is a norm of {n.d}, rows have {d}")
    mod = None
    parts = [t for t in (gate, scale, shift) if t is not None]
    if parts:
        rows = parts[0].shape[0]
        lds = [_matrix(t, (rows, d), _BF16, "gate, scale or shift", dev)[1] for t in parts]
        if len(set(lds)) > 1:
            raise OQError(OQ_ERR_INVALID_ARG, f"gate, scale and shift must have one row stride, got {lds}")
        mod = ctypes.byref(oq_mod(*(None if t is None else t.data_ptr() for t in (gate, scale, shift)),
                                  _opt(row, T, _I32, "row", dev), lds[0], rows))
    _check(_lib.oq_residual_norm(y_at, y_ld, k, _opt(weights, T * k, _F, "weights", dev), y_scale, r_at, r_ld, r_scale, _TYPES[r_type],
                                 T, d, None if post is None else _wide(post, dev, "post"),
                                 None if pre is None else _wide(pre, dev, "pre"), mod, ro_at, ro_ld, h_at, h_ld, stream))
    return (r_out if want_r else None), (h if want_h else None)


def oq_logprobs_ws_bytes(T: int, V: int, n: int, top: int) -> int:
    """Scratch bytes of one call; fewer rows can take more than more do."""
    _small(V, n, top)
    return int(_lib.oq_logprobs_ws_bytes(T, V, n, top))


def oq_logprobs(logits, tokens=None, top: int = 0, scale: float = 1.0, logprob=None, rank=None, entropy=None, lse=None, top_id=None,
                top_logprob=None, ws=None):
    """logits float32 or bfloat16 [T][V]; tokens int32 [T][n] (None: n = 0); returns
    (logprob [T][n], rank [T][n], entropy [T], lse [T], top_id [T][top], top_logprob [T][top])."""
    dev, stream, dtype, at, ld = _logits(logits, "logits")
    T, V = logits.shape
    n = 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != T:
            raise OQError(OQ_ERR_INVALID_ARG, f"tokens must be a matrix of {T} rows")
        n = tokens.shape[1]
    _small(V, n, top)

    new, device = torch.empty, logits.device

    def out(t, shape, count, dtype, what):
        """(tensor, address) of an output, allocated where none is given."""
        if t is None:
            t = new(shape, dtype=dtype, device=device)
            return t, t.data_ptr()
        return t, _vec(t, count, dtype, what, dev)

    top_n = max(top, 0)
    logprob, logprob_at = out(logprob, (T, n), T * n, _F, "logprob")
    rank, rank_at = out(rank, (T, n), T * n, _I32, "rank")
    entropy, entropy_at = out(entropy, (T,), T, _F, "entropy")
    lse, lse_at = out(lse, (T,), T, _F, "lse")
    top_id, id_at = out(top_id, (T, top_n), T * top_n, _I32, "top_id")
    top_logprob, top_at = out(top_logprob, (T, top_n), T * top_n, _F, "top_logprob")
    ws, ws_at, ws_bytes = _scratch(ws, lambda: oq_logprobs_ws_bytes(T, V, n, top), dev, device)
    _check(_lib.oq_logprobs(at, dtype, ld, T, V, scale, _opt(tokens, T * n, _I32, "tokens", dev), n, top, logprob_at, rank_at, entropy_at,
                            lse_at, id_at, top_at, ws_at, ws_bytes, stream))
    return logprob, rank, entropy, lse, top_id, top_logprob
