"""What stands around and inside the MoE layer's products (oracle; test
infrastructure only): token int8 codes and the int8 product, the gated
feed-forward block with its recomputing backward, and the norms around a block.

Float64 everywhere, except the codec steps (fp32 by definition), the int8
product's scales (fp32 by definition, so that its bf16 result is exact) and the
stored bf16 A.
"""
from __future__ import annotations

import numpy as np

from .ckpt import ckpt_save, swiglu_bwd_values, swiglu_from_values
from .codecs import FMT_INT8, FMT_NONE, fq_act
from .numerics import bf16_to_f32, f32_to_bf16, f64_to_bf16


def quantize_tokens(x_bits):
    """bf16 bits [rows, K] -> (codes uint8 [rows, K], scale fp32 [rows]): one
    checkpoint group a row."""
    codes, scale = ckpt_save(x_bits, FMT_INT8, np.asarray(x_bits).shape[1])
    return codes, scale[:, 0]


def _segments(seg):
    return [(e, int(seg[e]), int(seg[e + 1])) for e in range(len(seg) - 1) if seg[e + 1] > seg[e]]


def _rows(perm, topk, r0, r1):
    return np.arange(r0, r1) if perm is None else np.asarray(perm, np.int64)[r0:r1] // topk


def int8_sums(xc, sx, perm, topk, seg, wc, sw):
    """fp32 (sum_k cx cw) * sx * sw for every routed row [seg[-1], N]; wc uint8
    [E, N, K], sw [E, N] or [E]."""
    x = np.asarray(xc, np.uint8).view(np.int8).astype(np.float64)
    w = np.asarray(wc, np.uint8).view(np.int8)
    out = np.zeros((int(seg[-1]), w.shape[1]), np.float32)
    for e, r0, r1 in _segments(seg):
        rows = _rows(perm, topk, r0, r1)
        acc = x[rows] @ w[e].astype(np.float64).T          # integers below 2^53: exact
        with np.errstate(all="ignore"):
            out[r0:r1] = (acc.astype(np.float32) * np.asarray(sx, np.float32)[rows][:, None]) \
                * np.asarray(sw, np.float32)[e]
    return out


def gemm_int8(xc, sx, perm, topk, seg, wc, sw):
    """bf16 bits [seg[-1], N]."""
    return f32_to_bf16(int8_sums(xc, sx, perm, topk, seg, wc, sw))


def gated_sums(x_bits, perm, topk, seg, w_bits):
    """h = [g, u] of every routed row, float64 [seg[-1], 2F]."""
    x = bf16_to_f32(x_bits).astype(np.float64)
    w = bf16_to_f32(w_bits).astype(np.float64)
    out = np.zeros((int(seg[-1]), w.shape[1]))
    for e, r0, r1 in _segments(seg):
        out[r0:r1] = x[_rows(perm, topk, r0, r1)] @ w[e].T
    return out


def gated(h, afmt=FMT_NONE, act_scale=None):
    """(bf16 bits of FQ_a(A), A's bits) from h [R, 2F]."""
    a = f64_to_bf16(swiglu_from_values(h)[3])
    return (a if afmt == FMT_NONE else fq_act(a, afmt, act_scale).bits), a


def gated_bwd(daq, h, afmt=FMT_NONE, act_scale=None):
    """float64 dh [R, 2F] from daq [R, F] (values) and h."""
    a = f64_to_bf16(swiglu_from_values(h)[3])
    m = 1.0 if afmt == FMT_NONE else fq_act(a, afmt, act_scale).mask
    return swiglu_bwd_values(np.asarray(daq, np.float64) * m, h)


def rms(v, eps):
    """1 / sqrt(mean(v^2) + eps) of every row, [T, 1]."""
    v = np.asarray(v, np.float64)
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def norm_residual(x, b, gate, alpha, w_post, w_pre, eps):
    """(y, n) in float64; n None without w_pre."""
    y = np.asarray(x, np.float64)
    if b is not None:
        p = np.asarray(b, np.float64)
        if w_post is not None:
            p = p * rms(b, eps) * w_post
        if gate is not None:
            p = p * np.asarray(gate, np.float64)[:, None]
        y = y + alpha * p
    return y, None if w_pre is None else y * rms(y, eps) * w_pre


def norm_residual_bwd(dy, dn, y, b, gate, alpha, w_post, w_pre, eps):
    """dict of dx, db, dgate, dw_post, dw_pre in float64 (those that exist)."""
    y = np.asarray(y, np.float64)
    H = y.shape[1]
    gy = np.zeros_like(y) if dy is None else np.asarray(dy, np.float64).copy()
    out = {}
    if dn is not None:
        r = rms(y, eps)
        v = np.asarray(dn, np.float64) * w_pre
        gy += r * v - y * r ** 3 * ((v * y).sum(1, keepdims=True) / H)
        out["dw_pre"] = (dn * y * r).sum(0)
    out["dx"] = gy
    if b is None:
        return out
    b = np.asarray(b, np.float64)
    rb = rms(b, eps) if w_post is not None else 1.0
    w = np.ones(H) if w_post is None else np.asarray(w_post, np.float64)
    q = alpha * (np.ones(len(y)) if gate is None else np.asarray(gate, np.float64))[:, None]
    if gate is not None:
        out["dgate"] = alpha * (gy * b * rb * w).sum(1)
    dp = q * gy
    if w_post is None:
        out["db"] = dp
        return out
    out["dw_post"] = (dp * b * rb).sum(0)
    v = dp * w
    out["db"] = rb * v - b * rb ** 3 * ((v * b).sum(1, keepdims=True) / H)
    return out
