"""Pins of the 8-bit activation checkpoints' oracle, and the library's refusals
of bad checkpoint calls (no GPU needed)."""
import numpy as np
import pytest
import torch

import oracle as O
from test_abi_host import _no_gpu_visible, pkg  # noqa: F401  (fixture)

host_only = pytest.mark.skipif(not _no_gpu_visible(), reason="placeholder pointers")

FMTS = [O.FMT_INT8, O.FMT_FP8]


def _x(rows, K, seed=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal(K))
    return O.f32_to_bf16(x.astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [16, 64, 512])
def test_error_is_at_most_half_a_step(fmt, group):
    """|x - x~| <= s/2 (int8); E4M3: half a step of its binade, at least 2^-10 of s."""
    bits = _x(9, 1024)
    x = O.bf16_to_f32(bits).astype(np.float64)
    codes, s = O.ckpt_save(bits, fmt, group)
    v = O.ckpt_values(codes, s, fmt).astype(np.float64)
    sg = np.repeat(s.astype(np.float64), group, axis=1)
    z = np.abs(x / sg)
    # z and code * s are each rounded once to fp32: three relative 2^-24
    slack = 3 * 2.0 ** -24 * np.abs(x)
    if fmt == O.FMT_INT8:
        half = 0.5
    else:
        half = 2.0 ** (np.floor(np.log2(np.maximum(z, 2.0 ** -6))) - 4)
    assert np.all(np.abs(v - x) <= half * sg + slack)
    # the group's largest magnitude maps to the last code
    top = np.abs(codes.view(np.int8).astype(int)) if fmt == O.FMT_INT8 else codes & 0x7F
    assert np.all(top.reshape(9, -1, group).max(-1) == (127 if fmt == O.FMT_INT8 else 0x7E))


@pytest.mark.parametrize("fmt", FMTS)
def test_special_groups(fmt):
    bits = np.zeros((5, 16), np.uint16)
    bits[1, :] = 0x0001                  # the smallest subnormal
    bits[2, 3] = 0x7F80                  # an infinity
    bits[3, 5] = 0xFFC1                  # a NaN
    bits[4, :] = 0x7F7F                  # the largest finite value
    codes, s = O.ckpt_save(bits, fmt, 16)
    v = O.ckpt_values(codes, s, fmt)
    assert s[0, 0] == 1 and np.all(codes[0] == 0) and np.all(v[0] == 0)
    assert s[1, 0] == np.float32(2.0 ** -126) and np.all(np.abs(v[1]) <= 2.0 ** -126)
    assert np.isnan(s[2, 0]) and np.all(codes[2] == 0) and np.all(np.isnan(v[2]))
    assert np.isnan(s[3, 0]) and np.all(codes[3] == 0) and np.all(np.isnan(v[3]))
    assert np.all(np.isfinite(v[4])) and np.all(v[4] > 3.3e38)


def test_saved_twice_is_saved_once():
    """Loaded values whose scale is a power of two save to the same codes."""
    rng = np.random.default_rng(3)
    codes = rng.integers(-127, 128, (4, 64)).astype(np.int8)
    codes[:, ::32] = 127
    s = np.full((4, 2), 2.0 ** -5, np.float32)
    bits = O.ckpt_load(codes.view(np.uint8), s, O.FMT_INT8)
    c2, s2 = O.ckpt_save(bits, O.FMT_INT8, 32)
    assert np.array_equal(c2.view(np.int8), codes) and np.array_equal(s2, s)


def test_swiglu_gradient_against_autograd_and_differences():
    rng = np.random.default_rng(4)
    h = rng.standard_normal((3, 64)) * 2
    da = rng.standard_normal((3, 32))
    dh = O.swiglu_bwd_values(da, h)
    t = torch.from_numpy(h).requires_grad_(True)
    (torch.nn.functional.silu(t[:, :32]) * t[:, 32:] * torch.from_numpy(da)).sum().backward()
    assert np.allclose(dh, t.grad.numpy(), rtol=1e-12, atol=1e-13)
    eps = 1e-5
    for j in rng.choice(64, 8, replace=False):
        hp, hm = h.copy(), h.copy()
        hp[:, j] += eps
        hm[:, j] -= eps
        num = ((O.swiglu_from_values(hp)[3] - O.swiglu_from_values(hm)[3]) * da).sum(1) / (2 * eps)
        # central differences: eps^2/6 times a third derivative below 4 |da| |u|, plus cancellation
        assert np.all(np.abs(num - dh[:, j]) <= 1e-8 * (1 + np.abs(da).sum(1)))


@host_only
def test_refusals(pkg):  # noqa: F811
    lib, P = pkg.lib(), 0x1000
    aq = pkg.fq_act_q(pkg.FMT_NONE, None)
    import ctypes
    ref = ctypes.byref(aq)

    def save(x=P, rows=4, K=256, fmt=pkg.FMT_INT8, group=64, codes=P, scale=P):
        return lib.fq_ckpt_save(x, rows, K, None, fmt, group, codes, scale, None)

    def load(x=P, rows=4, K=256, fmt=pkg.FMT_INT8, group=64, codes=P, scale=P):
        return lib.fq_ckpt_load(codes, scale, rows, K, None, fmt, group, x, None)

    for call in (save, load):
        for bad in (dict(x=None), dict(codes=None), dict(scale=None), dict(rows=-1), dict(K=0),
                    dict(K=24), dict(fmt=pkg.FMT_NVFP4), dict(fmt=pkg.FMT_INT4), dict(fmt=0),
                    dict(group=0), dict(group=8), dict(group=48), dict(group=1024, K=1024),
                    dict(group=512), dict(group=-1), dict(x=P + 2), dict(codes=P + 8),
                    dict(scale=P + 2), dict(rows=1 << 30, K=256)):
            assert call(**bad) == pkg.FQ_ERR_INVALID_ARGUMENT, (call.__name__, bad)
            assert lib.fq_last_error()

    def fwd(h=P, R=4, n=P, F=128, q=ref, fmt=pkg.FMT_INT8, group=64, a=None, aqo=P, codes=P,
            scale=P):
        return lib.fq_swiglu_actfq_ckpt(h, R, n, F, q, fmt, group, a, aqo, codes, scale, None)

    def bwd(h=P, R=4, n=P, F=128, q=ref, fmt=pkg.FMT_INT8, group=64, a=None, aqo=P, codes=P,
            scale=P, ds=None, ws=None, wsb=0):
        return lib.fq_swiglu_bwd_ckpt(h, codes, scale, R, n, F, fmt, group, q, aqo, a, ds, ws, wsb,
                                      None)

    noscale = pkg.fq_act_q(pkg.FMT_FP8_E4M3, None)
    for call in (fwd, bwd):
        for bad in (dict(h=None), dict(n=None), dict(aqo=None), dict(codes=None), dict(scale=None),
                    dict(F=120), dict(F=0), dict(F=-16), dict(R=-1), dict(fmt=pkg.FMT_NVFP4),
                    dict(group=256), dict(group=32, F=48), dict(h=P + 4), dict(a=P + 4),
                    dict(q=ctypes.byref(noscale)), dict(R=1 << 27, F=128)):
            assert call(**bad) == pkg.FQ_ERR_INVALID_ARGUMENT, (call.__name__, bad)
    # a learnable scale needs fp8 / int8 activations and a workspace
    assert bwd(ds=P) == pkg.FQ_ERR_UNSUPPORTED
    q8 = ctypes.byref(pkg.fq_act_q(pkg.FMT_FP8_E4M3, P))
    assert bwd(ds=P, q=q8) == pkg.FQ_ERR_WORKSPACE_TOO_SMALL
