"""The few-token MoE layer rounds neither A without an activation format nor
weights of small groups: a case of integers whose outputs are small differences
of large A, and the oracle on it (no GPU needed)."""
import numpy as np
import pytest

import oracle as O
from tokens_case import reference

FORMS = [(O.FMT_INT4, 128), (O.FMT_INT4, 32), (O.FMT_INT4, None), (O.FMT_INT8, None),
         (O.FMT_INT8, 64), (O.FMT_INT8, O.GROUP_TENSOR), (O.FMT_FP8, 16), (O.FMT_FP8, None),
         (O.FMT_NVFP4, 16), (O.FMT_NONE, 0)]


def difference_case(seed, T, E, H, F, fmt, group, uneven=False):
    """Gates near 100, where silu(g) = g in fp32, ups near 150, all integers; the
    channels i and i + F/2 differ by 1 in their ups, and every row of W_d takes
    one such difference: out = +-g, exactly, from two A of 14 bits. uneven: the
    channels' scales are 0.9 and 1.1 bf16 half steps above 1, in both stacks, so
    that products rounded to bf16 are off by 2^-8 against each other."""
    rng = np.random.default_rng(seed)
    small = lambda *s: rng.integers(-1, 2, s) * (rng.random(s) < 0.2)  # noqa: E731
    gate, up = small(E, F // 2, H), small(E, F // 2, H)
    gate[..., :3], up[..., :3] = 0, 0
    gate[..., 0], up[..., 1] = 1, 1
    gu = np.concatenate([gate, gate, up, up], 1).astype(np.float32)
    gu[:, F + F // 2:, 2] = 1.0
    d = np.zeros((E, H, F), np.float32)
    pick, sign = rng.integers(0, F // 2, (E, H)), rng.choice([-1.0, 1.0], (E, H))
    for k, s in ((0, 1), (F // 2, -1)):
        np.put_along_axis(d, (pick + k)[..., None], (s * sign)[..., None].astype(np.float32), 2)
    x = rng.integers(0, 3, (T, H)).astype(np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 100, 150, 1

    def scales(N, K, stack):
        g = K if group is None else group
        if fmt == O.FMT_NONE:
            return None, None, None
        if group == O.GROUP_TENSOR:
            return np.ones(E, np.float32), None, None
        s = np.ones((E, N, K // g), np.float32)
        if uneven:
            s[:] = 1 + 0.9 * 2.0 ** -8
            high = s.reshape(E, 2, 2, F // 2, -1)[:, :, 1] if stack == "gu" else s[..., F // 2 // g:]
            high[:] = 1 + 1.1 * 2.0 ** -8
        return (s, np.full_like(s, 8) if fmt == O.FMT_INT4 else None,
                np.ones(E, np.float32) if fmt == O.FMT_NVFP4 else None)

    return dict(T=T, E=E, H=H, F=F, topk=1, afmt=O.FMT_NONE, begin=0, x=O.f32_to_bf16(x),
                ids=rng.integers(0, E, (T, 1)).astype(np.int32), probs=np.ones((T, 1), np.float32),
                gu=(fmt, H if group is None else group, O.f32_to_bf16(gu), scales(2 * F, H, "gu")),
                d=(fmt, F if group is None else group, O.f32_to_bf16(d), scales(H, F, "d")),
                s1=np.float32(1), s2=np.float32(1))


def by_definition(c, hold=lambda a: a, hold_w=lambda w: w):
    """The layer from its definition in float64, A and the weights held as
    `hold` and `hold_w` make them. (Every weight is a code times its scale.)"""
    gu, d = (O.bf16_to_f32(c[k][2]).astype(np.float64) for k in ("gu", "d"))
    if c["gu"][3][0] is not None and c["gu"][3][0].ndim == 3:
        gu, d = (w * np.repeat(s.astype(np.float64), w.shape[2] // s.shape[2], axis=2)
                 for w, s in ((gu, c["gu"][3][0]), (d, c["d"][3][0])))
    gu, d = hold_w(gu), hold_w(d)
    x, F = O.bf16_to_f32(c["x"]).astype(np.float64), c["F"]
    out = np.zeros((c["T"], c["H"]))
    for t in range(c["T"]):
        e = int(c["ids"][t, 0])
        h = gu[e] @ x[t]
        assert 40 <= h[:F].min() and np.abs(h).max() < 250
        out[t] = d[e] @ hold(h[:F] / (1.0 + np.exp(-h[:F])) * h[F:])
    return out


def _bf16(a):
    return O.bf16_to_f32(O.f64_to_bf16(a)).astype(np.float64)


@pytest.mark.parametrize("fmt,group", FORMS)
def test_a_is_not_rounded(fmt, group):
    """Two bf16 parts of A give the outputs, one does not."""
    c = difference_case(7, 5, 3, 256, 256, fmt, group)
    ref, tol = reference(c)
    want = by_definition(c)
    # the bound: h off by (H + 36) 2^-24 of sums of magnitudes below 400, each of two A by
    # 2.1 x 250 of that, and 550 2^-24 of two magnitudes below 62500: 11.4
    assert np.all(np.abs(want) >= 40) and np.all(tol < 11.4)
    assert np.allclose(ref, want, rtol=0, atol=1e-9)
    assert np.all(np.abs(by_definition(c, lambda a: _bf16(a) + _bf16(a - _bf16(a))) - ref) <= tol)
    one = np.abs(by_definition(c, _bf16) - ref)
    assert np.mean(one > tol + 2.0 ** -8 * (np.abs(ref) + tol)) > 0.5


SMALL_GROUPS = [(O.FMT_INT8, 16), (O.FMT_INT8, 32), (O.FMT_FP8, 16), (O.FMT_FP8, 32),
                (O.FMT_INT4, 32), (O.FMT_INT4, 64)]


@pytest.mark.parametrize("fmt,group", SMALL_GROUPS)
def test_weights_of_small_groups_are_not_rounded(fmt, group):
    """Two bf16 parts of each weight give the outputs, one does not."""
    c = difference_case(8, 5, 3, 256, 256, fmt, group, uneven=True)
    ref, tol = reference(c)
    two = lambda v: _bf16(v) + _bf16(v - _bf16(v))  # noqa: E731
    # the bound as above, and 2^-16 of the sums of magnitudes: h 2^-16 x 400 more, which
    # either A takes 1.1 x 500 of, and twice 3 x 2^-16 of two magnitudes below 64000
    assert np.all(tol < 11.4 + 6.8 + 11.8)
    assert np.allclose(ref, by_definition(c), rtol=0, atol=1e-9)
    assert np.all(np.abs(by_definition(c, two, two) - ref) <= tol)
    one = np.abs(by_definition(c, hold_w=_bf16) - ref)
    assert np.mean(one > tol + 2.0 ** -8 * (np.abs(ref) + tol)) > 0.5
