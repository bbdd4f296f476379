"""Pins of the oracle's token codes, int8 product, gated block and norms: against
torch's float64 autograd, central differences, integer arithmetic and closed forms."""
import numpy as np
import pytest
import torch

import oracle as O

EPS = 1e-6


def _bits(rng, *shape, std=1.0):
    return O.f32_to_bf16((rng.standard_normal(shape) * std).astype(np.float32))


def test_token_codes_closed_forms():
    x = np.zeros((7, 32), np.float32)
    x[1, 3], x[1, 4], x[1, 5] = 127.0, -63.5, 0.5      # s = 1: ties to even
    x[2] = np.ldexp(np.arange(-16, 16), -140)           # at most 2^-136: bf16 rounds it to zero
    x[6] = np.ldexp(np.arange(-16, 16), -131)           # subnormals: the floor of s
    x[3, 0], x[4, 0], x[5, :] = np.inf, np.nan, -2.0
    codes, s = O.quantize_tokens(O.f32_to_bf16(x))
    c = codes.view(np.int8)
    assert s[0] == 1.0 and not c[0].any()
    assert abs(float(s[1]) - 1.0) < 1e-7 and c[1, 3] == 127 and c[1, 4] == -64 and c[1, 5] == 0
    assert s[2] == 1.0 and not c[2].any()
    assert s[6] == np.float32(2.0 ** -126)
    assert np.isnan(s[3]) and np.isnan(s[4]) and not c[3].any() and not c[4].any()
    assert np.all(c[5] == -127)


def test_token_codes_are_within_half_a_step():
    rng = np.random.default_rng(0)
    b = _bits(rng, 40, 96)
    codes, s = O.quantize_tokens(b)
    v = O.bf16_to_f32(b).astype(np.float64)
    err = np.abs(codes.view(np.int8) * s[:, None].astype(np.float64) - v)
    assert np.all(err <= s[:, None] * (0.5 + 2.0 ** -16))
    assert np.all(np.abs(codes.view(np.int8)).max(1) == 127)


def test_int8_product_against_python_integers():
    rng = np.random.default_rng(1)
    E, N, K, T, topk = 3, 16, 32, 5, 2
    xc = rng.integers(-128, 128, (T, K)).astype(np.int8).view(np.uint8)
    wc = rng.integers(-128, 128, (E, N, K)).astype(np.int8).view(np.uint8)
    sx = rng.random(T).astype(np.float32)
    perm = np.array([3, 0, 9, 4], np.int32)
    seg = np.array([0, 1, 1, 4], np.int32)
    for sw in (rng.random((E, N)).astype(np.float32), rng.random(E).astype(np.float32)):
        got = O.int8_sums(xc, sx, perm, topk, seg, wc, sw)
        for r, e in ((0, 0), (1, 2), (2, 2), (3, 2)):
            t = int(perm[r]) // topk
            for n in range(N):
                acc = sum(int(a) * int(b) for a, b in zip(xc[t].view(np.int8), wc[e, n].view(np.int8)))
                s = sw[e, n] if sw.ndim == 2 else sw[e]
                assert got[r, n] == np.float32(np.float32(acc) * sx[t]) * s


@pytest.mark.parametrize("afmt,as_", [(O.FMT_NONE, 1.0), (O.FMT_FP8, 0.003), (O.FMT_INT8, 0.01)])
def test_gated_backward_against_autograd(afmt, as_):
    rng = np.random.default_rng(2)
    E, H, Fc, T, topk = 2, 32, 16, 6, 2
    x, w = _bits(rng, T, H), _bits(rng, E, 2 * Fc, H, std=0.3)
    perm = np.array([1, 4, 11, 0, 7], np.int32)
    seg = np.array([0, 2, 5], np.int32)
    h = O.gated_sums(x, perm, topk, seg, w)
    d = rng.standard_normal((5, Fc))
    th = torch.tensor(h, requires_grad=True)
    a = torch.nn.functional.silu(th[:, :Fc]) * th[:, Fc:]
    _, ab = O.gated(h)
    m = 1.0 if afmt == O.FMT_NONE else O.fq_act(ab, afmt, as_).mask
    if afmt != O.FMT_NONE:
        assert 0.02 < 1.0 - m.mean() < 0.98       # the mask matters here
    (a * torch.tensor(d * m)).sum().backward()
    assert np.allclose(th.grad.numpy(), O.gated_bwd(d, h, afmt, as_), rtol=1e-12, atol=1e-14)
    # rows through perm / topk, by hand
    xv, wv = O.bf16_to_f32(x).astype(np.float64), O.bf16_to_f32(w).astype(np.float64)
    for r in range(5):
        assert np.allclose(h[r], wv[0 if r < 2 else 1] @ xv[perm[r] // topk], rtol=1e-14)


CASES = [dict(), dict(gate=False), dict(post=False), dict(post=False, gate=False), dict(block=False),
         dict(pre=False), dict(pre=False, post=False)]


def _norm_inputs(rng, T, H, block=True, gate=True, post=True, pre=True):
    g = rng.standard_normal
    return dict(x=g((T, H)), b=g((T, H)) if block else None, gate=g(T) if block and gate else None,
                w_post=1 + 0.3 * g(H) if block and post else None, w_pre=1 + 0.3 * g(H) if pre else None)


@pytest.mark.parametrize("kw", CASES)
def test_norm_backward_against_autograd_and_differences(kw):
    rng = np.random.default_rng(3)
    T, H, alpha = 4, 16, 0.7
    inp = _norm_inputs(rng, T, H, **kw)
    dy, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    if inp["w_pre"] is None:
        dn = None
    t = {k: torch.tensor(v, requires_grad=True) for k, v in inp.items() if v is not None}
    y = t["x"] * 1.0
    if "b" in t:
        p = t["b"]
        if "w_post" in t:
            p = p * torch.rsqrt(p.square().mean(1, keepdim=True) + EPS) * t["w_post"]
        if "gate" in t:
            p = p * t["gate"][:, None]
        y = y + alpha * p
    loss = (y * torch.tensor(dy)).sum()
    if "w_pre" in t:
        n = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * t["w_pre"]
        loss = loss + (n * torch.tensor(dn)).sum()
    loss.backward()
    ry, rn = O.norm_residual(inp["x"], inp["b"], inp["gate"], alpha, inp["w_post"], inp["w_pre"], EPS)
    assert np.allclose(ry, y.detach().numpy(), rtol=1e-12)
    if rn is not None:
        assert np.allclose(rn, n.detach().numpy(), rtol=1e-12)
    got = O.norm_residual_bwd(dy, dn, ry, inp["b"], inp["gate"], alpha, inp["w_post"], inp["w_pre"], EPS)
    names = dict(x="dx", b="db", gate="dgate", w_post="dw_post", w_pre="dw_pre")
    for k, v in t.items():
        assert np.allclose(got[names[k]], v.grad.numpy(), rtol=1e-9, atol=1e-12), k

    def value(z):
        a, c = O.norm_residual(z["x"], z["b"], z["gate"], alpha, z["w_post"], z["w_pre"], EPS)
        return (a * dy).sum() + (0.0 if c is None else (c * dn).sum())

    for k in t:
        d = rng.standard_normal(inp[k].shape)
        up, dn_ = dict(inp), dict(inp)
        up[k], dn_[k] = inp[k] + 1e-5 * d, inp[k] - 1e-5 * d
        slope = (value(up) - value(dn_)) / 2e-5
        want = (got[names[k]] * d).sum()
        # central differences: 1e-10 of curvature and 1e-16 / 1e-5 of rounding, of sums of ~100
        assert abs(slope - want) <= 1e-6 * (1 + abs(want)), k


def test_norm_of_a_zero_row_is_zero_and_its_gradient_finite():
    H = 16
    y, n = O.norm_residual(np.zeros((1, H)), np.zeros((1, H)), None, 1.0, np.ones(H), np.ones(H), EPS)
    assert not y.any() and not n.any()
    got = O.norm_residual_bwd(np.ones((1, H)), np.ones((1, H)), y, np.zeros((1, H)), None, 1.0,
                              np.ones(H), np.ones(H), EPS)
    assert np.allclose(got["dx"], 1.0 + 1e3) and np.allclose(got["db"], 1e3 * got["dx"])
    assert not got["dw_pre"].any() and not got["dw_post"].any()
