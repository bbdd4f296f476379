"""GPU parity of the norms around a block, forward and backward, against float64."""
import numpy as np
import pytest
import torch

import oracle as O
from block_case import normal_bits
from helpers import bf16_vals, dev_bf16, dev_f32, host_bits
from test_gpu_graph import _capture

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

EPS, ALPHA, FILL = 1e-6, 0.7, 7.0
U = 2.0 ** -24      # half a step of fp32
SHAPES = [(1, 16), (3, 48), (130, 512), (5, 528), (9, 2048), (2, 2064), (1, 4096), (7, 8192), (3, 8208),
          (2, 16384), (2100, 64)]
FORMS = [dict(), dict(gate=False), dict(post=False), dict(post=False, gate=False), dict(block=False),
         dict(pre=False), dict(pre=False, post=False)]


class Case:
    def __init__(self, T, H, seed, block=True, gate=True, post=True, pre=True):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.rng = T, H, rng
        self.x = normal_bits(rng, T, H) if T * H else np.zeros((T, H), np.uint16)
        if T > 2:
            self.x[0] = 0                                     # rows of zeros
        self.b = normal_bits(rng, T, H, std=3.0) if block else None
        if T > 2 and block:
            self.b[0] = self.b[1] = 0
        self.gate = rng.standard_normal(T).astype(np.float32) if block and gate else None
        self.w_post = O.f32_to_bf16((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)) if block and post else None
        self.w_pre = O.f32_to_bf16((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)) if pre else None

    def vals(self):
        v = lambda t: None if t is None else bf16_vals(t)  # noqa: E731
        return (v(self.b), self.gate, ALPHA_F, v(self.w_post), v(self.w_pre), EPS_F)

    def dev(self):
        d = lambda t: None if t is None else dev_bf16(t)  # noqa: E731
        return (d(self.b), None if self.gate is None else dev_f32(self.gate), ALPHA, d(self.w_post),
                d(self.w_pre), EPS, self.T, self.H)


ALPHA_F, EPS_F = float(np.float32(ALPHA)), float(np.float32(EPS))


def bf16_out(*shape):
    return torch.full(shape, FILL, dtype=torch.bfloat16, device="cuda")


def _fwd_errors(c, y, n):
    """How far fp32 takes y and n from float64: a mean of squares is within
    (H + 8) U of itself, its root half of that, then a few products."""
    x = bf16_vals(c.x)
    k = (c.H / 2 + 12) * U
    ey = k * np.abs(y - x) + 2 * U * np.abs(y)
    if n is None:
        return ey, None
    ry = O.blocks.rms(y, EPS_F)
    w = np.abs(bf16_vals(c.w_pre))
    # y's own error reaches n through its element and through the mean
    through = np.sqrt((ey * ey).mean(1, keepdims=True)) * ry
    return ey, k * np.abs(n) + ey * ry * w + 1.01 * through * np.abs(n)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("form", FORMS)
def test_forward(T, H, form):
    print(f"[norm] T={T} H={H} {form}", flush=True)
    c = Case(T, H, T + H, **form)
    y, n = O.norm_residual(bf16_vals(c.x), *c.vals())
    ey, en = _fwd_errors(c, y, n)
    gy, gn = bf16_out(T, H), bf16_out(T, H) if n is not None else None
    F.fq_norm_residual_fwd(dev_bf16(c.x), *c.dev(), gy, gn)
    assert np.all(np.abs(bf16_vals(host_bits(gy)) - y) <= 2.0 ** -8 * np.abs(y) + ey * 1.01)
    if n is None:
        return
    assert np.all(np.abs(bf16_vals(host_bits(gn)) - n) <= 2.0 ** -8 * np.abs(n) + en * 1.01)
    # n alone, and its codes with the same n, give the same n
    n2, n3 = bf16_out(T, H), bf16_out(T, H)
    codes = torch.full((T, H), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((T,), -3.0, device="cuda")
    F.fq_norm_residual_fwd(dev_bf16(c.x), *c.dev(), None, n2)
    F.fq_norm_residual_fwd(dev_bf16(c.x), *c.dev(), None, n3, codes, s)
    assert torch.equal(gn, n2) and torch.equal(gn, n3)
    q, sv = codes.cpu().numpy().view(np.int8).astype(np.float64), s.cpu().numpy().astype(np.float64)
    amax = np.abs(n).max(1)
    want = np.where(amax == 0, 1.0, np.maximum(amax / 127, 2.0 ** -126))
    assert np.all(np.abs(sv - want) <= (en.max(1) / 127 + 3 * U * want))
    # a code stands for n within half a step, the step's rounding (codes up to 128) and n's error
    assert np.all(np.abs(q * sv[:, None] - n) <= sv[:, None] * (0.5 + 300 * U) + en * 1.01)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("form", FORMS)
def test_backward(T, H, form):
    print(f"[norm bwd] T={T} H={H} {form}", flush=True)
    c = Case(T, H, 3 * T + H, **form)
    pre = c.w_pre is not None
    dy_b, dn_b = normal_bits(c.rng, T, H), normal_bits(c.rng, T, H) if pre else None
    x, dy, dn = bf16_vals(c.x), bf16_vals(dy_b), bf16_vals(dn_b) if pre else None
    ref = O.norm_residual_bwd(dy, dn, x, *c.vals())
    b, gate, alpha, w_post, w_pre, eps = c.vals()
    out = dict(dx=bf16_out(T, H))
    if b is not None:
        out["db"] = bf16_out(T, H)
    if gate is not None:
        out["dgate"] = torch.full((T,), FILL, device="cuda")
    if w_post is not None:
        out["dw_post"] = torch.full((H,), FILL, device="cuda")
    if pre:
        out["dw_pre"] = torch.full((H,), FILL, device="cuda")
    ws = torch.empty(max(256, F.fq_workspace_bytes(F.FQ_OP_NORM, (1, T, H), 0, 0)), dtype=torch.uint8,
                     device="cuda")
    args = (dev_bf16(dy_b), dev_bf16(dn_b) if pre else None, dev_bf16(c.x), *c.dev())
    F.fq_norm_residual_bwd(*args, **out, ws=ws)
    got = {k: bf16_vals(host_bits(v)) if v.dtype == torch.bfloat16 else v.cpu().numpy().astype(np.float64)
           for k, v in out.items()}
    # sums over a row: (H + 8) U of their magnitudes; the roots' errors beside them
    k = (2 * H + 40) * U
    mag = np.abs(dy)
    if pre:
        r = O.blocks.rms(x, eps)
        v = np.abs(dn * w_pre)
        mag = mag + r * v + np.abs(x) * r ** 3 * (v * np.abs(x)).mean(1, keepdims=True)
    e_gy = k * mag
    assert np.all(np.abs(got["dx"] - ref["dx"]) <= 2.0 ** -8 * np.abs(ref["dx"]) + 1.01 * e_gy)
    if pre:
        t = np.abs(dn * x * r)
        assert np.all(np.abs(got["dw_pre"] - ref["dw_pre"]) <= 1.01 * (k + (T + 32) * U) * t.sum(0))
    if b is None:
        return
    rb = O.blocks.rms(b, eps) if w_post is not None else 1.0
    w = np.ones(H) if w_post is None else np.abs(w_post)
    q = alpha * (1.0 if gate is None else np.abs(gate)[:, None].astype(np.float64)) * np.ones((T, 1))
    gmag = mag + e_gy           # every term that gy's magnitude and error bring
    if gate is not None:
        t = alpha * (gmag * np.abs(b) * rb * w).sum(1)
        assert np.all(np.abs(got["dgate"] - ref["dgate"]) <= 1.01 * 2 * k * t)
    if w_post is None:
        assert np.all(np.abs(got["db"] - ref["db"]) <= 2.0 ** -8 * np.abs(ref["db"]) + 1.01 * 2 * k * q * gmag)
    else:
        m = q * (rb * gmag * w + np.abs(b) * rb ** 3 * (gmag * w * np.abs(b)).mean(1, keepdims=True))
        assert np.all(np.abs(got["db"] - ref["db"]) <= 2.0 ** -8 * np.abs(ref["db"]) + 1.01 * 3 * k * m)
        t = (q * gmag * np.abs(b) * rb).sum(0)
        assert np.all(np.abs(got["dw_post"] - ref["dw_post"]) <= 1.01 * (2 * k + (T + 32) * U) * t)
    # each output alone has the same bits, and so has one without the weights' sums
    for name in out:
        alone = torch.full_like(out[name], FILL)
        F.fq_norm_residual_bwd(*args, **{name: alone}, ws=ws)
        assert torch.equal(alone, out[name]), name


def test_one_gradient_alone_and_in_place():
    """dy or dn missing; y over x, dx over dy or dn, db over b."""
    T, H = 70, 272
    c = Case(T, H, 1)
    x, dy, dn = dev_bf16(c.x), dev_bf16(normal_bits(c.rng, T, H)), dev_bf16(normal_bits(c.rng, T, H))
    b, rest = c.dev()[0], c.dev()[1:]
    zero = torch.zeros_like(dy)
    y, n, y2, n2 = (bf16_out(T, H) for _ in range(4))
    F.fq_norm_residual_fwd(x, b, *rest, y, n)
    over = x.clone()
    F.fq_norm_residual_fwd(over, b, *rest, over, n2)
    assert torch.equal(over, y) and torch.equal(n, n2)
    for d1, d2 in ((dy, None), (None, dn), (dy, dn)):
        dx, db, dx2, db2 = (bf16_out(T, H) for _ in range(4))
        F.fq_norm_residual_bwd(d1, d2, y, b, *rest, dx=dx, db=db)
        F.fq_norm_residual_bwd(zero if d1 is None else d1, zero if d2 is None else d2, y, b, *rest, dx=dx2,
                               db=db2)
        assert torch.equal(dx, dx2) and torch.equal(db, db2)
        o1 = (d1 if d1 is not None else d2).clone()
        b1 = b.clone()
        F.fq_norm_residual_bwd(o1 if d1 is not None else None, o1 if d1 is None else d2, y, b1, *rest, dx=o1,
                               db=b1)
        assert torch.equal(o1, dx) and torch.equal(b1, db)


def test_no_tokens():
    F.fq_norm_residual_fwd(None, None, None, 1.0, None, dev_bf16(np.zeros(32, np.uint16)), EPS, 0, 32, None,
                           bf16_out(1, 32))
    dw, dp = torch.full((32,), FILL, device="cuda"), torch.full((32,), FILL, device="cuda")
    w = dev_bf16(np.zeros(32, np.uint16))
    F.fq_norm_residual_bwd(None, None, None, bf16_out(1, 32), None, 1.0, w, w, EPS, 0, 32, dw_pre=dw, dw_post=dp)
    assert not dw.any() and not dp.any()


def test_a_row_that_is_not_finite_stays_alone():
    T, H = 9, 80
    c = Case(T, H, 2)
    c.x[4, 7] = 0x7FC0
    c.b[6, 0] = 0x7F80
    y, n = bf16_out(T, H), bf16_out(T, H)
    codes, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(T, device="cuda")
    F.fq_norm_residual_fwd(dev_bf16(c.x), *c.dev(), y, n, codes, s)
    ok = [t for t in range(T) if t not in (4, 6)]
    assert torch.isfinite(y[ok].float()).all() and torch.isfinite(n[ok].float()).all()
    assert torch.isfinite(s[ok]).all() and torch.isnan(s[[4, 6]]).all() and not codes[[4, 6]].any()


def test_replays_and_another_stream():
    T, H = 333, 1040
    c = Case(T, H, 6)
    x, dn = dev_bf16(c.x), dev_bf16(normal_bits(c.rng, T, H))
    dev = c.dev()

    def bufs():
        f = lambda n: torch.full((n,), FILL, device="cuda")  # noqa: E731
        return dict(y=bf16_out(T, H), n=bf16_out(T, H), dx=bf16_out(T, H), db=bf16_out(T, H), dgate=f(T),
                    dw_post=f(H), dw_pre=f(H),
                    ws=torch.empty(F.fq_workspace_bytes(F.FQ_OP_NORM, (1, T, H), 0, 0), dtype=torch.uint8,
                                   device="cuda"))

    def step(o):
        F.fq_norm_residual_fwd(x, *dev, o["y"], o["n"])
        F.fq_norm_residual_bwd(o["n"], dn, o["y"], *dev, **{k: o[k] for k in
                               ("dx", "db", "dgate", "dw_post", "dw_pre", "ws")})

    one, two, cap = bufs(), bufs(), bufs()
    step(one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(two)
    step(one)
    torch.cuda.synchronize()
    names = [k for k in one if k != "ws"]
    assert all(torch.equal(one[k], two[k]) for k in names)
    g = _capture(lambda: step(cap))
    for rep in range(3):
        x.copy_(dev_bf16(normal_bits(c.rng, T, H)))
        for k in names:
            cap[k].fill_(FILL)
        g.replay()
        step(one)
        torch.cuda.synchronize()
        assert all(torch.equal(one[k], cap[k]) for k in names), f"replay {rep}"
