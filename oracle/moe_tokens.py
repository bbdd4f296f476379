"""A whole MoE layer over stored weights for a few tokens (oracle; test
infrastructure only): float64 from the definition, with a bound on what fp32
arithmetic may change.

h = W_gu FQ_a1(x), a = silu(h_g) h_u in full precision, A = FQ_a2(a) (a itself
without an activation format), out[t] = sum over the local slots of p W_d A.

The bound: an fp32 sum of n products in any order is off by at most
(n + 32) 2^-24 times the sum of the magnitudes; that moves a, and the
quantizer maps the moved interval onto grid values (an interval that crosses a
rounding border takes the values of both sides). Without an activation format
the other side may hold A as two bf16 numbers, A rounded (off by at most half a
step, 2^-8 |A|) and the rest rounded (2^-8 of that): 2^-16 |A| in all, or half
the smallest subnormal step, and a sum of twice as many products. It may hold
weights of small groups (stored_values' bf16 ones) alike, and leave out the
product of the two rests, again 2^-16 of the whole: up to three products an element.
"""
from __future__ import annotations

import numpy as np

from .codecs import (FMT_FP8, FMT_INT4, FMT_INT8, FMT_NONE, FMT_NVFP4, E2M1_MAX, E4M3_MAX,
                     e2m1_round, e4m3_round, fq_act, fq_weight_stack)
from .moe import _sigmoid
from .numerics import bf16_to_f32

U = 2.0 ** -24


class _Decoded(np.ndarray):
    """A decoded stack whose values are bf16 numbers; exact: before the rounding."""

    exact = None


def _exact(w):
    """A stack's values, and the bf16 parts that the other side may take them in."""
    e = getattr(w, "exact", None)
    return (np.asarray(w), 1) if e is None else (e, 2)


def stored_values(w_bits, fmt: int, group: int, scale, zp=None, g=None):
    """float64 values of a stored stack [E, N, K]: value(code) * scale, or the
    bf16 fake-quant value (as fq_dequantize_stacked gives it) where the group is
    smaller than 64 (int8, fp8) or not a multiple of 128 (int4) and not the whole
    row. The layer multiplies with the values before that rounding."""
    fq = fq_weight_stack(w_bits, fmt, group, scale, zp, g)
    if fmt == FMT_NONE:
        return fq.v.astype(np.float64)
    E, N, K = fq.q.shape
    if fmt == FMT_NVFP4:
        th = e4m3_round(np.clip(scale, 0, E4M3_MAX).astype(np.float32))[1]
        s = np.repeat(th, 16, axis=-1) * np.asarray(g, np.float64).reshape(E, 1, 1)
    elif group < 0:
        s = np.asarray(scale, np.float64).reshape(E, 1, 1)
    else:
        s = np.repeat(np.asarray(scale, np.float64).reshape(E, N, K // group), group, axis=-1)
    v = fq.q * s
    if fmt in (FMT_INT8, FMT_FP8, FMT_INT4) and 0 < group < K \
            and group % (128 if fmt == FMT_INT4 else 64):
        v, exact = bf16_to_f32(fq.bits).astype(np.float64).view(_Decoded), v
        v.exact = exact
    return v


def _quant(a, fmt, s, theta=None):
    """FQ_a of fp32 rows on a given NVFP4 theta (else its own), float64 values."""
    a = np.asarray(a, np.float32)
    s = np.float32(s)
    if fmt == FMT_NVFP4:
        sb = (theta * s).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            z = (a * (np.float32(1) / sb).astype(np.float32)).astype(np.float32)
        z = np.where(sb == 0, np.float32(0), z)
        return e2m1_round(np.clip(z, -E2M1_MAX, E2M1_MAX))[1] * theta.astype(np.float64) * float(s)
    z = (a * (np.float32(1) / s)).astype(np.float32)
    if fmt == FMT_FP8:
        return e4m3_round(z)[1] * float(s)
    return np.rint(np.clip(z, -128, 127)).astype(np.float64) * float(s)


def _theta(amax, s):
    r = (np.float32(1) / (np.float32(6) * np.float32(s))).astype(np.float32)
    t = np.minimum((amax.astype(np.float32) * r).astype(np.float32), np.float32(E4M3_MAX))
    return e4m3_round(t)[1].astype(np.float32)


def quant_interval(lo, mid, hi, fmt, s):
    """FQ_a(mid) and the largest distance from it that a value between lo and
    hi (elementwise) may be quantized to."""
    if fmt == FMT_NONE:
        return mid, np.maximum(hi - mid, mid - lo) + 2.0 ** -16 * np.abs(mid) + 2.0 ** -134
    if fmt != FMT_NVFP4:
        v = _quant(mid, fmt, s)
        return v, np.maximum(np.abs(_quant(lo, fmt, s) - v), np.abs(_quant(hi, fmt, s) - v))
    b = [x.reshape(x.shape[0], -1, 16) for x in (lo, mid, hi)]
    top = np.maximum(np.abs(b[0]), np.abs(b[2])).max(-1)
    bot = np.where((b[0] <= 0) & (b[2] >= 0), 0.0, np.minimum(np.abs(b[0]), np.abs(b[2]))).max(-1)
    th = _theta(np.abs(b[1]).max(-1), s)
    exp = lambda t: np.repeat(t, 16, axis=-1).reshape(mid.shape)  # noqa: E731
    v = _quant(mid, fmt, s, exp(th))
    d = np.zeros_like(v)
    # theta is monotone in the block's amax, and it moves by at most one step here
    for t in (th, _theta(bot, s), _theta(top, s)):
        for x in (lo, mid, hi):
            d = np.maximum(d, np.abs(_quant(x, fmt, s, exp(t)) - v))
    return v, d


def moe_tokens(x_bits, ids, probs, ebegin: int, w_gu, w_d, afmt: int, s1, s2, rel_h: float = 0.0,
               afmt2=None):
    """out [T, H] float64 and its tolerance before the rounding to bf16.
    w_gu [E, 2F, H], w_d [E, H, F]: stored_values. rel_h: a further relative
    error of h and of a that the other side may have. afmt2: A's activation
    format where it is not x's."""
    T = len(ids)
    E, F2, H = w_gu.shape
    F = F2 // 2
    (w_gu, parts_gu), (w_d, parts_d) = _exact(w_gu), _exact(w_d)
    afmt2 = afmt if afmt2 is None else afmt2
    fx = fq_act(x_bits, afmt, s1)
    xq = fx.q * float(np.float32(s1)) if afmt in (FMT_FP8, FMT_INT8) else fx.v.astype(np.float64)
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(np.asarray(ids[t]) - ebegin):
            if not 0 <= e < E:
                continue
            p = float(probs[t, j])
            h = w_gu[e] @ xq[t]
            # the scales outside the sum and the NVFP4 block scale's own rounding: 4 more
            dh = ((parts_gu * H + 36) * U + (parts_gu - 1) * 2.0 ** -16) \
                * (np.abs(w_gu[e]) @ np.abs(xq[t])) + rel_h * np.abs(h)
            g, u = h[:F], h[F:]
            sg = _sigmoid(g)
            a = g * sg * u
            # |silu'| <= 1.1; sigmoid's own error as |g| 2^-23 and a few ulp
            da = (1.1 * dh[:F] * (np.abs(u) + dh[F:]) + np.abs(g * sg) * dh[F:]
                  + np.abs(a) * ((np.abs(g) + 10) * 2 * U + rel_h))
            A, dA = quant_interval((a - da)[None], a[None], (a + da)[None], afmt2, s2)
            A, dA = A[0], dA[0] + 4 * U * np.abs(A[0])
            o = w_d[e] @ A
            mag = np.abs(w_d[e]) @ np.abs(A)
            parts_a = 2 if afmt2 == FMT_NONE else 1
            two = (parts_d - 1) * parts_a * 2.0 ** -16
            tol[t] += abs(p) * (np.abs(w_d[e]) @ dA + rel_h * np.abs(o)
                                + (((parts_d + parts_a - 1) * F + 36) * U + two) * mag)
            out[t] += p * o
    return out, tol + 80 * U * np.abs(out)
