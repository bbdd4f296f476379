"""Activation checkpoints in 8 bits (oracle; test infrastructure only).

A row of K elements is kept as one byte per element with an fp32 scale per
group: s = max(fp32(amax * fp32(1/D)), 2^-126) with D = 127 (int8) or 448
(E4M3), 1 for an all-zero group; r = fp32(1 / s); code = Q(clamp(fp32(x * r))); loaded
value code * s. A group with an infinity or NaN has s = NaN and codes 0.

The SwiGLU backward from a checkpoint takes g, u as the fp32 values code * s;
everything after that is float64 here, except that A is stored as bf16 and the
activation quantizer's steps are fp32 by definition.
"""
from __future__ import annotations

import numpy as np

from .codecs import FMT_FP8, FMT_INT8, e4m3_round, e4m3_value_of_code
from .moe import _sigmoid
from .numerics import bf16_to_f32, f32_to_bf16, f64_to_bf16

CKPT_D = {FMT_INT8: np.float32(127.0), FMT_FP8: np.float32(448.0)}


def ckpt_save(x_bits, fmt: int, group: int):
    """bf16 bits [rows, K] -> (codes uint8 [rows, K], scale fp32 [rows, K/group])."""
    x = bf16_to_f32(x_bits)
    rows, K = x.shape
    b = x.reshape(rows, K // group, group)
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(-1)
        inv = np.float32(1) / CKPT_D[fmt]
        s = np.maximum((amax * inv).astype(np.float32), np.float32(2.0 ** -126))
        s = np.where(amax == 0, np.float32(1), s).astype(np.float32)
        bad = ~np.isfinite(amax)
        r = np.where(bad, np.float32(0), np.float32(1) / s).astype(np.float32)
        z = np.where(bad[..., None], np.float32(0), (b * r[..., None]).astype(np.float32))
    if fmt == FMT_INT8:
        codes = np.rint(np.clip(z, -128.0, 127.0)).astype(np.int8).view(np.uint8)
    else:
        codes = e4m3_round(z)[0]
    codes = np.where(bad[..., None], np.uint8(0), codes)
    return codes.reshape(rows, K), np.where(bad, np.float32(np.nan), s).astype(np.float32)


def ckpt_values(codes, scale, fmt: int):
    """The fp32 values code * s, [rows, K]."""
    codes = np.asarray(codes, np.uint8)
    rows, K = codes.shape
    v = codes.view(np.int8).astype(np.float32) if fmt == FMT_INT8 \
        else e4m3_value_of_code(codes).astype(np.float32)
    s = np.asarray(scale, np.float32)
    with np.errstate(invalid="ignore"):
        return (v.reshape(rows, s.shape[1], -1) * s[..., None]).astype(np.float32).reshape(rows, K)


def ckpt_load(codes, scale, fmt: int):
    """bf16 bits of the loaded tensor (a NaN group: NaN, any payload)."""
    return f32_to_bf16(ckpt_values(codes, scale, fmt))


def swiglu_from_values(h):
    """float64 g, u, sigmoid(g) and A = silu(g) u of h [R, 2F] (fp32 values)."""
    h = np.asarray(h, np.float64)
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s = _sigmoid(g)
    return g, u, s, g * s * u


def swiglu_bwd_values(da, h):
    """float64 dh [R, 2F] of A = silu(g) u for an upstream da [R, F]."""
    g, u, s, _ = swiglu_from_values(h)
    da = np.asarray(da, np.float64)
    return np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], 1)


def a_bits_of(h):
    """The stored A: bf16 bits of silu(g) u."""
    return f64_to_bf16(swiglu_from_values(h)[3])
