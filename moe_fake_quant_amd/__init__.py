"""Python binding of libfq, the gfx950 C-ABI library for scale-only fake-quant
MoE grouped GEMM (argument marshalling only: every step runs in libfq's HIP
kernels; torch provides device memory and the current stream).

Each function has the name and argument order of its C entry point in
include/fq.h, takes device tensors (or None for a NULL pointer), enqueues on
``torch.cuda.current_stream()`` and raises ``FQError`` for a non-OK status.
Importing this package loads ``libfq.so`` and ``_fqbind.so`` (the native
marshalling of the calls whose kernels are short) from this directory and fails
loudly when one is missing; there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfq.so")

FQ_OK = 0
FQ_ERR_INVALID_ARGUMENT = 1
FQ_ERR_UNSUPPORTED = 2
FQ_ERR_WORKSPACE_TOO_SMALL = 3
FQ_ERR_HIP = 4

FMT_NONE = 0
FMT_INT8 = 1
FMT_INT4 = 2
FMT_FP8_E4M3 = 3
FMT_NVFP4 = 4
FMT_BY_NAME = {"none": FMT_NONE, "int8": FMT_INT8, "int4": FMT_INT4, "fp8": FMT_FP8_E4M3,
               "nvfp4": FMT_NVFP4}

FQ_OP_PERMUTE = 1
FQ_OP_GEMM_FWD = 2
FQ_OP_GEMM_BWD = 3
FQ_OP_ACT_SCALE_GRAD = 4
FQ_OP_TOPK_KL = 5
FQ_OP_MOE_TOKENS = 6
FQ_OP_GEMM_INT8 = 7
FQ_OP_GATED = 8
FQ_OP_NORM = 9
FQ_GROUP_TENSOR = -1     # one weight scale per expert matrix (int8 / fp8)

EXPORTED = (
    "observer_absmax_init", "fq_quantize_stacked", "fq_moe_permute", "fq_grouped_gemm_fwd",
    "fq_grouped_gemm_bwd_scale", "fq_moe_gather_actfq", "fq_swiglu_actfq", "fq_swiglu_bwd",
    "fq_moe_combine", "fq_moe_combine_bwd", "fq_moe_unpermute_reduce", "fq_workspace_bytes",
    "fq_last_error", "fq_abi_version", "fq_export_scales", "fq_dequantize_stacked", "fq_topk_kl",
    "fq_moe_permute_noalloc", "fq_validate", "fq_actfq", "fq_grouped_gemm_fwd_tokens",
    "fq_grouped_gemm_wgrad_tokens", "fq_ckpt_save", "fq_ckpt_load", "fq_swiglu_actfq_ckpt",
    "fq_swiglu_bwd_ckpt", "fq_moe_tokens", "fq_quantize_tokens", "fq_grouped_gemm_int8",
    "fq_grouped_gated_int8", "fq_grouped_gated_fwd", "fq_grouped_gated_bwd", "fq_norm_residual_fwd",
    "fq_norm_residual_bwd",
)

FQ_BAD_EXPERT_ID = 0x01
FQ_BAD_SEG_START = 0x02
FQ_BAD_SEG_ORDER = 0x04
FQ_BAD_SEG_END = 0x08
FQ_BAD_SCALE = 0x10
FQ_BAD_ZERO_POINT = 0x20
FQ_BAD_GLOBAL_SCALE = 0x40
FQ_BAD_ACT_SCALE = 0x80


class FQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libfq status {status}: {msg}")
        self.status = status


class fq_shape(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32)]


class fq_weight_q(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("group", ctypes.c_int32), ("scale", ctypes.c_void_p),
                ("zero_point", ctypes.c_void_p), ("global_scale", ctypes.c_void_p)]


class fq_act_q(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("scale", ctypes.c_void_p)]


class fq_stored_w(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("group", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("scale_bytes", ctypes.c_void_p),
                ("zero_point_bytes", ctypes.c_void_p), ("global_scale", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfq.so not found at {LIB_PATH}; build it with "
                          "`python moe_fake_quant_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    F32 = ctypes.c_float
    st = ctypes.c_int
    sig = {
        "observer_absmax_init": (st, [P, fq_shape, I32, I32, I32, P, P, P, P, SZ, P]),
        "fq_quantize_stacked": (st, [P, fq_shape, ctypes.POINTER(fq_weight_q), P, P, P]),
        "fq_moe_permute": (st, [P, I32, I32, I32, I32, P, P, P, P, SZ, P]),
        "fq_moe_permute_noalloc": (st, [P, I32, I32, I32, I32, P, P, P, P]),
        "fq_validate": (st, [P, I32, I32, I32, P, I32, I32, fq_shape, ctypes.POINTER(fq_weight_q),
                             ctypes.POINTER(fq_act_q), P, P]),
        "fq_grouped_gemm_fwd": (st, [P, I32, P, fq_shape, P, P, ctypes.POINTER(fq_weight_q),
                                     ctypes.POINTER(fq_act_q), P, P, SZ, P]),
        "fq_grouped_gemm_bwd_scale": (st, [P, P, I32, P, fq_shape, P, P,
                                           ctypes.POINTER(fq_weight_q), ctypes.POINTER(fq_act_q),
                                           P, P, P, P, SZ, P]),
        "fq_actfq": (st, [P, I32, I32, ctypes.POINTER(fq_act_q), P, P]),
        "fq_grouped_gemm_fwd_tokens": (st, [P, I32, P, I32, I32, P, fq_shape, P, P,
                                            ctypes.POINTER(fq_weight_q), P, P, SZ, P]),
        "fq_grouped_gemm_wgrad_tokens": (st, [P, P, I32, P, I32, I32, P, fq_shape, P,
                                              ctypes.POINTER(fq_weight_q), P, P, P, SZ, P]),
        "fq_moe_gather_actfq": (st, [P, I32, I32, P, I32, ctypes.POINTER(fq_act_q), P, P]),
        "fq_swiglu_actfq": (st, [P, I32, P, I32, ctypes.POINTER(fq_act_q), P, P, P]),
        "fq_swiglu_bwd": (st, [P, P, I32, P, I32, ctypes.POINTER(fq_act_q), P, P, P, SZ, P]),
        "fq_moe_combine": (st, [P, P, P, I32, I32, I32, P, P]),
        "fq_moe_combine_bwd": (st, [P, P, P, I32, I32, I32, P, P]),
        "fq_moe_unpermute_reduce": (st, [P, P, P, I32, I32, I32, ctypes.POINTER(fq_act_q), P, P,
                                         P, SZ, P]),
        "fq_export_scales": (st, [fq_shape, ctypes.POINTER(fq_weight_q), P, P, P]),
        "fq_dequantize_stacked": (st, [P, fq_shape, I32, I32, P, P, P, P, P, P]),
        "fq_topk_kl": (st, [P, P, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P]),
        "fq_moe_tokens": (st, [P, I32, I32, I32, P, P, I32, I32, I32, ctypes.POINTER(fq_stored_w),
                               ctypes.POINTER(fq_stored_w), ctypes.POINTER(fq_act_q),
                               ctypes.POINTER(fq_act_q), P, P, SZ, P]),
        "fq_ckpt_save": (st, [P, I32, I32, P, I32, I32, P, P, P]),
        "fq_ckpt_load": (st, [P, P, I32, I32, P, I32, I32, P, P]),
        "fq_swiglu_actfq_ckpt": (st, [P, I32, P, I32, ctypes.POINTER(fq_act_q), I32, I32, P, P, P,
                                      P, P]),
        "fq_swiglu_bwd_ckpt": (st, [P, P, P, I32, P, I32, I32, I32, ctypes.POINTER(fq_act_q), P, P,
                                    P, P, SZ, P]),
        "fq_quantize_tokens": (st, [P, I32, I32, P, P, P, P]),
        "fq_grouped_gemm_int8": (st, [P, P, I32, P, I32, I32, P, fq_shape,
                                      ctypes.POINTER(fq_stored_w), P, P, SZ, P]),
        "fq_grouped_gated_int8": (st, [P, P, I32, P, I32, I32, P, fq_shape,
                                       ctypes.POINTER(fq_stored_w), P, P, SZ, P]),
        "fq_grouped_gated_fwd": (st, [P, I32, P, I32, I32, P, fq_shape, P, ctypes.POINTER(fq_act_q), P,
                                      P, SZ, P]),
        "fq_grouped_gated_bwd": (st, [P, P, I32, P, I32, I32, P, fq_shape, P, ctypes.POINTER(fq_act_q),
                                      P, P, P, SZ, P]),
        "fq_norm_residual_fwd": (st, [P, P, P, F32, P, P, F32, I32, I32, P, P, P, P, P]),
        "fq_norm_residual_bwd": (st, [P, P, P, P, P, F32, P, P, F32, I32, I32, P, P, P, P, P, P, SZ,
                                      P]),
        "fq_workspace_bytes": (SZ, [I32, fq_shape, I32, I32]),
        "fq_last_error": (ctypes.c_char_p, []),
        "fq_abi_version": (I32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()

from . import _fqbind as _b  # noqa: E402  (built next to libfq.so, which it links)


def lib() -> ctypes.CDLL:
    return _lib


def abi_version() -> int:
    return _lib.fq_abi_version()


def _check(status: int):
    if status != FQ_OK:
        raise FQError(status, _lib.fq_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libfq takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libfq takes contiguous tensors")
    return t.data_ptr()


# The current stream's handle without a Stream object around it: 0.2 us instead
# of 2.8 us of every call's 7.3 us on the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _same_device(t: Optional[torch.Tensor]):
    """The calls run on the current device's stream; its kernels must not be
    handed another device's memory."""
    if t is not None and t.is_cuda and t.get_device() != torch.cuda.current_device():
        raise ValueError(f"tensor on cuda:{t.get_device()}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


@dataclasses.dataclass
class WeightQ:
    """Weight quantizer: fmt, group, scale [E,N,K/group] (nvfp4: theta),
    zero_point (int4), global_scale [E] (nvfp4)."""
    fmt: int
    group: int
    scale: Optional[torch.Tensor] = None
    zero_point: Optional[torch.Tensor] = None
    global_scale: Optional[torch.Tensor] = None

    def c(self) -> fq_weight_q:
        return fq_weight_q(self.fmt, self.group, _p(self.scale), _p(self.zero_point),
                           _p(self.global_scale))


@dataclasses.dataclass
class ActQ:
    """Activation quantizer: fmt and a one-element device scale (s_a or g_a)."""
    fmt: int = FMT_NONE
    scale: Optional[torch.Tensor] = None

    def c(self) -> fq_act_q:
        return fq_act_q(self.fmt, _p(self.scale))


@dataclasses.dataclass
class StoredW:
    """A weight stack in its stored (exported) form: fmt, group, codes
    [E,N,K] packed (fmt NONE: the bf16 stack), and the format's scales."""
    fmt: int
    group: int = 0
    codes: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None
    scale_bytes: Optional[torch.Tensor] = None
    zero_point_bytes: Optional[torch.Tensor] = None
    global_scale: Optional[torch.Tensor] = None

    def c(self) -> fq_stored_w:
        return fq_stored_w(self.fmt, self.group, _p(self.codes), _p(self.scale),
                           _p(self.scale_bytes), _p(self.zero_point_bytes), _p(self.global_scale))


def _shape(E, N, K) -> fq_shape:
    return fq_shape(int(E), int(N), int(K))


def _aq(aq: Optional[ActQ]):
    return ctypes.byref(aq.c()) if aq is not None else None


def _nbytes(ws: Optional[torch.Tensor]) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def fq_workspace_bytes(op: int, shape, R_max: int, fmts: int) -> int:
    return int(_lib.fq_workspace_bytes(op, _shape(*shape), int(R_max), int(fmts)))


def observer_absmax_init(x, shape, fmt, group, per_tensor, scale, zero_point=None,
                         global_scale=None, ws=None):
    _check(_lib.observer_absmax_init(_p(x), _shape(*shape), fmt, group, int(per_tensor), _p(scale),
                                     _p(zero_point), _p(global_scale), _p(ws), _nbytes(ws),
                                     _stream()))


def fq_quantize_stacked(w, shape, q: WeightQ, w_fq=None, codes=None):
    _check(_lib.fq_quantize_stacked(_p(w), _shape(*shape), ctypes.byref(q.c()), _p(w_fq),
                                    _p(codes), _stream()))


def fq_moe_permute(expert_ids, T, topk, expert_begin, E_local, perm, row_of, seg_offsets, ws):
    _check(_lib.fq_moe_permute(_p(expert_ids), int(T), int(topk), int(expert_begin),
                               int(E_local), _p(perm), _p(row_of), _p(seg_offsets), _p(ws),
                               _nbytes(ws), _stream()))


def fq_moe_permute_noalloc(expert_ids, T, topk, expert_begin, E_local, perm, row_of,
                           seg_offsets):
    _check(_lib.fq_moe_permute_noalloc(_p(expert_ids), int(T), int(topk), int(expert_begin),
                                       int(E_local), _p(perm), _p(row_of), _p(seg_offsets),
                                       _stream()))


def fq_validate(status, expert_ids=None, T=0, topk=0, n_experts=0, seg_offsets=None, E=0,
                R_max=0, shape=(1, 1, 1), wq: Optional[WeightQ] = None, aq: Optional[ActQ] = None):
    """Enqueue the device-data checks; `status` (one int32/uint32 device
    element) receives the OR of the FQ_BAD_* bits of failed conditions."""
    _check(_lib.fq_validate(_p(expert_ids), int(T), int(topk), int(n_experts), _p(seg_offsets),
                            int(E), int(R_max), _shape(*shape),
                            ctypes.byref(wq.c()) if wq is not None else None,
                            ctypes.byref(aq.c()) if aq is not None else None, _p(status),
                            _stream()))


def fq_grouped_gemm_fwd(x, R_max, seg_offsets, shape, w, w_fq, wq: Optional[WeightQ],
                        aq: Optional[ActQ], y, ws=None):
    _check(_lib.fq_grouped_gemm_fwd(_p(x), int(R_max), _p(seg_offsets), _shape(*shape), _p(w),
                                    _p(w_fq), ctypes.byref(wq.c()) if wq is not None else None,
                                    _aq(aq), _p(y), _p(ws),
                                    _nbytes(ws), _stream()))


def fq_grouped_gemm_bwd_scale(dy, x, R_max, seg_offsets, shape, w, w_fq, wq: WeightQ,
                              aq: Optional[ActQ], dx, dscale, dzero_point=None, ws=None):
    _check(_lib.fq_grouped_gemm_bwd_scale(_p(dy), _p(x), int(R_max), _p(seg_offsets),
                                          _shape(*shape), _p(w), _p(w_fq), ctypes.byref(wq.c()),
                                          _aq(aq), _p(dx), _p(dscale), _p(dzero_point), _p(ws),
                                          _nbytes(ws), _stream()))


def fq_actfq(x, rows, K, aq: Optional[ActQ], xq):
    _check(_lib.fq_actfq(_p(x), int(rows), int(K), _aq(aq), _p(xq), _stream()))


def fq_grouped_gemm_fwd_tokens(x_tok, T, perm, topk, R_max, seg_offsets, shape, w, w_fq,
                               wq: Optional[WeightQ], y, ws=None):
    _check(_lib.fq_grouped_gemm_fwd_tokens(_p(x_tok), int(T), _p(perm), int(topk), int(R_max),
                                           _p(seg_offsets), _shape(*shape), _p(w), _p(w_fq),
                                           ctypes.byref(wq.c()) if wq is not None else None,
                                           _p(y), _p(ws), _nbytes(ws), _stream()))


def fq_grouped_gemm_wgrad_tokens(dy, x_tok, T, perm, topk, R_max, seg_offsets, shape, w,
                                 wq: WeightQ, dscale, dzero_point=None, ws=None):
    _check(_lib.fq_grouped_gemm_wgrad_tokens(_p(dy), _p(x_tok), int(T), _p(perm), int(topk),
                                             int(R_max), _p(seg_offsets), _shape(*shape), _p(w),
                                             ctypes.byref(wq.c()), _p(dscale), _p(dzero_point),
                                             _p(ws), _nbytes(ws), _stream()))


def fq_moe_gather_actfq(x, T, H, row_of, topk, aq: Optional[ActQ], xq):
    _check(_lib.fq_moe_gather_actfq(_p(x), int(T), int(H), _p(row_of), int(topk), _aq(aq),
                                    _p(xq), _stream()))


def fq_swiglu_actfq(h, R_max, n_rows, F, aq: Optional[ActQ], a, aq_out):
    _check(_lib.fq_swiglu_actfq(_p(h), int(R_max), _p(n_rows), int(F), _aq(aq), _p(a),
                                _p(aq_out), _stream()))


def fq_swiglu_bwd(daq, h, R_max, n_rows, F, aq: Optional[ActQ], dh, dscale_a=None, ws=None):
    _check(_lib.fq_swiglu_bwd(_p(daq), _p(h), int(R_max), _p(n_rows), int(F), _aq(aq), _p(dh),
                              _p(dscale_a), _p(ws), _nbytes(ws), _stream()))


def fq_moe_combine(o, probs, row_of, T, topk, H, out):
    _check(_lib.fq_moe_combine(_p(o), _p(probs), _p(row_of), int(T), int(topk), int(H), _p(out),
                               _stream()))


def fq_moe_combine_bwd(dout, probs, row_of, T, topk, H, dO):
    _check(_lib.fq_moe_combine_bwd(_p(dout), _p(probs), _p(row_of), int(T), int(topk), int(H),
                                   _p(dO), _stream()))


def fq_moe_unpermute_reduce(dxq, row_of, x, T, topk, H, aq: Optional[ActQ], dx, dscale_a=None,
                            ws=None):
    _check(_lib.fq_moe_unpermute_reduce(_p(dxq), _p(row_of), _p(x), int(T), int(topk), int(H),
                                        _aq(aq), _p(dx), _p(dscale_a), _p(ws), _nbytes(ws),
                                        _stream()))


def fq_export_scales(shape, q: WeightQ, scale_bytes=None, zero_point_bytes=None):
    _check(_lib.fq_export_scales(_shape(*shape), ctypes.byref(q.c()), _p(scale_bytes),
                                 _p(zero_point_bytes), _stream()))


def fq_dequantize_stacked(codes, shape, fmt, group, w_bf16, scale=None, scale_bytes=None,
                          zero_point_bytes=None, global_scale=None):
    _check(_lib.fq_dequantize_stacked(_p(codes), _shape(*shape), int(fmt), int(group), _p(scale),
                                      _p(scale_bytes), _p(zero_point_bytes), _p(global_scale),
                                      _p(w_bf16), _stream()))


def fq_moe_tokens(x, T, H, F, expert_ids, probs, topk, expert_begin, E_local, w_gu: StoredW,
                  w_d: StoredW, aq1: Optional[ActQ], aq2: Optional[ActQ], out, ws=None):
    _same_device(x)
    _check(_lib.fq_moe_tokens(_p(x), int(T), int(H), int(F), _p(expert_ids), _p(probs), int(topk),
                              int(expert_begin), int(E_local), ctypes.byref(w_gu.c()),
                              ctypes.byref(w_d.c()), _aq(aq1), _aq(aq2), _p(out), _p(ws),
                              _nbytes(ws), _stream()))


def fq_ckpt_save(x, rows, K, n_rows, fmt, group, codes, scale):
    _same_device(x)
    _check(_lib.fq_ckpt_save(_p(x), int(rows), int(K), _p(n_rows), int(fmt), int(group), _p(codes),
                             _p(scale), _stream()))


def fq_ckpt_load(codes, scale, rows, K, n_rows, fmt, group, x):
    _same_device(codes)
    _check(_lib.fq_ckpt_load(_p(codes), _p(scale), int(rows), int(K), _p(n_rows), int(fmt),
                             int(group), _p(x), _stream()))


def fq_swiglu_actfq_ckpt(h, R_max, n_rows, F, aq: Optional[ActQ], fmt, group, a, aq_out, codes,
                         scale):
    _same_device(h)
    _check(_lib.fq_swiglu_actfq_ckpt(_p(h), int(R_max), _p(n_rows), int(F), _aq(aq), int(fmt),
                                     int(group), _p(a), _p(aq_out), _p(codes), _p(scale),
                                     _stream()))


def fq_swiglu_bwd_ckpt(daq, codes, scale, R_max, n_rows, F, fmt, group, aq: Optional[ActQ], dh,
                       aq_out=None, dscale_a=None, ws=None):
    _same_device(daq)
    _check(_lib.fq_swiglu_bwd_ckpt(_p(daq), _p(codes), _p(scale), int(R_max), _p(n_rows), int(F),
                                   int(fmt), int(group), _aq(aq), _p(dh), _p(aq_out), _p(dscale_a),
                                   _p(ws), _nbytes(ws), _stream()))


def fq_topk_kl(student, teacher, T, V, K, reverse, valid, topk_idx, grad, loss_tok, loss_mean, ws):
    _check(_lib.fq_topk_kl(_p(student), _p(teacher), int(T), int(V), int(K), int(bool(reverse)),
                           _p(valid), _p(topk_idx), _p(grad), _p(loss_tok), _p(loss_mean), _p(ws),
                           _nbytes(ws), _stream()))


# The calls below are marshalled natively (bind/bind.cpp): contiguous device tensors
# on the current device, of the C type's elements, or None; shape (E, N, K).

def fq_quantize_tokens(x, rows, K, n_rows, codes, scale):
    _check(_b.fq_quantize_tokens(x, rows, K, n_rows, codes, scale))


def fq_grouped_gemm_int8(x_codes, x_scale, x_rows, perm, topk, R_max, seg_offsets, shape, w: StoredW,
                         y, ws=None):
    _check(_b.fq_grouped_gemm_int8(x_codes, x_scale, x_rows, perm, topk, R_max, seg_offsets, shape, w,
                                   y, ws))


def fq_grouped_gated_int8(x_codes, x_scale, x_rows, perm, topk, R_max, seg_offsets, shape, w: StoredW,
                          a, ws=None):
    _check(_b.fq_grouped_gated_int8(x_codes, x_scale, x_rows, perm, topk, R_max, seg_offsets, shape, w,
                                    a, ws))


def fq_grouped_gated_fwd(x, x_rows, perm, topk, R_max, seg_offsets, shape, w_fq, aq: Optional[ActQ],
                         aq_out, ws=None):
    _check(_b.fq_grouped_gated_fwd(x, x_rows, perm, topk, R_max, seg_offsets, shape, w_fq, aq, aq_out,
                                   ws))


def fq_grouped_gated_bwd(daq, x, x_rows, perm, topk, R_max, seg_offsets, shape, w_fq,
                         aq: Optional[ActQ], dh, aq_out=None, ws=None):
    _check(_b.fq_grouped_gated_bwd(daq, x, x_rows, perm, topk, R_max, seg_offsets, shape, w_fq, aq, dh,
                                   aq_out, ws))


def fq_norm_residual_fwd(x, b, gate, alpha, w_post, w_pre, eps, T, H, y=None, n=None, codes=None,
                         scale=None):
    _check(_b.fq_norm_residual_fwd(x, b, gate, alpha, w_post, w_pre, eps, T, H, y, n, codes, scale))


def fq_norm_residual_bwd(dy, dn, y, b, gate, alpha, w_post, w_pre, eps, T, H, dx=None, db=None,
                         dgate=None, dw_post=None, dw_pre=None, ws=None):
    _check(_b.fq_norm_residual_bwd(dy, dn, y, b, gate, alpha, w_post, w_pre, eps, T, H, dx, db, dgate,
                                   dw_post, dw_pre, ws))


from .layer import MoEFakeQuantLayer  # noqa: E402,F401
from .block import MoEFakeQuantBlock  # noqa: E402,F401
