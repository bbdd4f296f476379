"""The norms' backward at the ends of its ranges, against float64: very large rows, the
smallest eps, and more rows than the grid has blocks."""
import numpy as np
import pytest
import torch

import oracle as O
from block_case import normal_bits
from helpers import bf16_vals, dev_bf16, dev_f32, host_bits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

U = 2.0 ** -24      # half a step of fp32
FILL = 7.0


def _bf16(v):
    return O.f32_to_bf16(np.asarray(v, np.float32))


def _weights(rng, H):
    return _bf16(1 + 0.3 * rng.standard_normal(H))


def _outputs(T, H, frozen=False):
    f = lambda *s, t=torch.float32: torch.full(s, FILL, dtype=t, device="cuda")  # noqa: E731
    out = dict(dx=f(T, H, t=torch.bfloat16), db=f(T, H, t=torch.bfloat16), dgate=f(T))
    if not frozen:
        out.update(dw_post=f(H), dw_pre=f(H))
    return out


def _run(dy, dn, y, b, gate, alpha, w_post, w_pre, eps, frozen=False):
    """The call with every gradient (frozen: without the weights'), as float64 arrays."""
    T, H = y.shape
    out = _outputs(T, H, frozen)
    ws = torch.empty(max(256, F.fq_workspace_bytes(F.FQ_OP_NORM, (1, T, H), 0, 0)), dtype=torch.uint8,
                     device="cuda")
    F.fq_norm_residual_bwd(None if dy is None else dev_bf16(dy), dev_bf16(dn), dev_bf16(y), dev_bf16(b),
                           dev_f32(gate), alpha, dev_bf16(w_post), dev_bf16(w_pre), eps, T, H, **out, ws=ws)
    return {k: bf16_vals(host_bits(v)) if v.dtype == torch.bfloat16 else v.cpu().numpy().astype(np.float64)
            for k, v in out.items()}


def _check(got, dy, dn, y, b, gate, alpha, w_post, w_pre, eps):
    """Each gradient within the fp32 steps of its formula: a sum over a row is within (H + 8)
    U of its magnitudes and a root within half of that, (2 H + 40) U for all that enters one
    value; a sum over the rows adds (T + 32) U; bf16 outputs half a step."""
    v = lambda t: None if t is None else bf16_vals(t)  # noqa: E731
    dy, dn, y, b, w_post, w_pre = (v(t) for t in (dy, dn, y, b, w_post, w_pre))
    T, H = y.shape
    ref = O.norm_residual_bwd(dy, dn, y, b, gate, alpha, w_post, w_pre, eps)
    k, kt = (2 * H + 40) * U, (T + 32) * U
    r, rb, w = O.blocks.rms(y, eps), O.blocks.rms(b, eps), np.abs(w_post)
    vy = np.abs(dn * w_pre)
    yr = np.abs(y) * r
    mag = r * (vy + yr * (vy * yr).mean(1, keepdims=True)) + (0.0 if dy is None else np.abs(dy))
    br = np.abs(b) * rb
    q = abs(alpha) * np.abs(gate)[:, None].astype(np.float64)
    gmag = mag * (1 + k)
    tol = dict(dx=2.0 ** -8 * np.abs(ref["dx"]) + 1.01 * k * mag,
               db=2.0 ** -8 * np.abs(ref["db"]) +
               1.01 * 3 * k * q * rb * (gmag * w + br * (gmag * w * br).mean(1, keepdims=True)),
               dgate=1.01 * 2 * k * abs(alpha) * (gmag * br * w).sum(1),
               dw_post=1.01 * (2 * k + kt) * (q * gmag * br).sum(0),
               dw_pre=1.01 * (k + kt) * np.abs(dn * yr).sum(0))
    for name, g in got.items():
        err = np.abs(g - ref[name])
        assert np.all(err <= tol[name]), (name, float((err / np.maximum(tol[name], 1e-300)).max()))


@pytest.mark.parametrize("H", [48, 528, 2064, 8192, 16384])
@pytest.mark.parametrize("size", [2.0 ** 46, 2.0 ** 53, 2.0 ** 56])
def test_rows_of_very_large_values(H, size):
    """dn as large as the rows, so that dx, of order one, is all the norm's: the sums of
    squares stay below 2^127 (3 * 2^14 * 2^112), the cube of the root far below 2^-149."""
    print(f"[norm large] H={H} size={size}", flush=True)
    T, rng = 7, np.random.default_rng(H)
    y, b, dn = (normal_bits(rng, T, H, std=size) for _ in range(3))
    args = (None, dn, y, b, rng.standard_normal(T).astype(np.float32), 0.5, _weights(rng, H), _weights(rng, H),
            1e-6)
    _check(_run(*args), *args)


@pytest.mark.parametrize("H", [48, 2064])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -126, 2.0 ** -90])
def test_the_smallest_eps_and_rows_of_zeros(H, eps):
    """A row of zeros has the root eps^-1/2 (up to 2^74.5): dx = dy + dn w_pre eps^-1/2
    there, and no NaN."""
    print(f"[norm eps] H={H} eps={eps}", flush=True)
    T, rng = 6, np.random.default_rng(H)
    y, b, dy = (normal_bits(rng, T, H) for _ in range(3))
    dn = normal_bits(rng, T, H, std=2.0 ** -40)
    y[1] = y[4] = b[2] = b[4] = 0
    args = (dy, dn, y, b, rng.standard_normal(T).astype(np.float32), 0.5, _weights(rng, H), _weights(rng, H), eps)
    _check(_run(*args), *args)


# rows of a wave (4096 in flight), of four waves (1024) and of eight and four waves (512): each
# block takes its second and its third row
@pytest.mark.parametrize("T,H", [(9001, 48), (8200, 512), (2500, 528), (2100, 2048), (1300, 2064), (1100, 4112),
                                 (1030, 8208)])
@pytest.mark.parametrize("post", [True, False])
def test_more_rows_than_blocks(T, H, post):
    print(f"[norm rows] T={T} H={H} post={post}", flush=True)
    rng = np.random.default_rng(T)
    y, b, dy, dn = (normal_bits(rng, T, H) for _ in range(4))
    y[::7], b[::11] = 0, 0
    gate = rng.standard_normal(T).astype(np.float32)
    args = (dy, dn, y, b, gate, 0.5, _weights(rng, H), _weights(rng, H), 1e-6)
    got = _run(*args)
    _check(got, *args)
    # and without the weights' sums, a block to every row
    frozen = _run(*args, frozen=True)
    assert all(np.array_equal(frozen[k], got[k]) for k in frozen)
    if post:
        return
    # without b every row ends at its first sum: one barrier a row
    out = dict(dx=torch.full((T, H), FILL, dtype=torch.bfloat16, device="cuda"),
               dw_pre=torch.full((H,), FILL, device="cuda"))
    ws = torch.empty(F.fq_workspace_bytes(F.FQ_OP_NORM, (1, T, H), 0, 0), dtype=torch.uint8, device="cuda")
    F.fq_norm_residual_bwd(dev_bf16(dy), dev_bf16(dn), dev_bf16(y), None, None, 1.0, None, dev_bf16(args[7]),
                           1e-6, T, H, **out, ws=ws)
    assert np.array_equal(bf16_vals(host_bits(out["dx"])), got["dx"])
    assert np.array_equal(out["dw_pre"].cpu().numpy().astype(np.float64), got["dw_pre"])
