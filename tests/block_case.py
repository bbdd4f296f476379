"""Inputs of the product and gated-block tests: routed rows with empty experts,
room behind the last row, and sums that every order of fp32 addition forms
exactly, so that only the sigmoid and the last rounding differ from float64."""
import numpy as np

import oracle as O


def route(rng, T, topk, E, skew=False, spare=0):
    """(perm, seg) of a random routing with empty experts; perm also holds `spare`
    pairs behind seg[E] that no row names."""
    P = T * topk
    live = P - spare
    w = rng.random(E)
    if E > 2:
        w[rng.integers(0, E)] = 0.0
        if skew:
            w[0] = 50.0
    e = rng.choice(E, live, p=w / w.sum())
    order = np.argsort(e, kind="stable")
    pairs = rng.permutation(P)
    perm = np.concatenate([pairs[:live][order], pairs[live:]]).astype(np.int32)
    seg = np.concatenate([[0], np.cumsum(np.bincount(e, minlength=E))]).astype(np.int32)
    return perm, seg


def exact_bits(rng, *shape, step=0.25, top=3):
    """bf16 values k * step, |k| <= top: products of two such tensors sum exactly in
    fp32 (top^2 * K < 2^24)."""
    return O.f32_to_bf16((rng.integers(-top, top + 1, shape) * step).astype(np.float32))


def normal_bits(rng, *shape, std=1.0):
    return O.f32_to_bf16((rng.standard_normal(shape) * std).astype(np.float32))


def codes(rng, *shape):
    return rng.integers(-128, 128, shape).astype(np.int8).view(np.uint8)


def a_bracket(h, dh=0.0):
    """bf16 bits that bound the stored A of h (float64) when g and u may each be off
    by dh and the sigmoid by (|g| + 8) 2^-23 of itself: the hardware exp carries
    |g| log2(e) 2^-24 from its argument, and a few ulp of it, the reciprocal and the
    products follow."""
    g, u, s, a = O.swiglu_from_values(h)
    # |d silu / dg| < 1.1
    err = np.abs(a) * (np.abs(g) + 8) * 2.0 ** -23 + dh * (1.1 * np.abs(u) + np.abs(g * s) + 1.1 * dh)
    return O.f64_to_bf16(a - err), O.f64_to_bf16(a + err), err
