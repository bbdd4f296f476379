"""GPU parity of the 8-bit activation checkpoints through the C ABI: codes,
scales and loaded values bit for bit, the SwiGLU forward equal to the plain
call, and the backward from the saved values against float64."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import ACT_DSCALE_TOL, bf16_vals, dev_bf16, dev_f32, dev_i32, host_bits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

FMTS = [O.FMT_INT8, O.FMT_FP8]
SHAPES = [(1, 16, 16), (1, 2048, 512), (3, 80, 16), (37, 1040, 16), (130, 192, 64), (5, 768, 256),
          (257, 96, 32), (64, 1024, 128)]


def _bits(rows, K, seed, specials=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal(K))
    b = O.f32_to_bf16(x.astype(np.float32))
    flat = b.reshape(-1)
    if specials and flat.size >= 1024:
        flat[0:16] = 0                       # an all-zero stretch
        flat[16:32] = 0x8000                 # negative zeros
        flat[32:48] = 0x0003                 # subnormals
        flat[48:64] = 0x7F7F
        flat[512] = 0x7F80                   # +inf
        flat[flat.size // 2 + 3] = 0xFFC0    # NaN
    return b


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K,group", SHAPES)
def test_save_and_load_bitexact(fmt, rows, K, group):
    print(f"[ckpt] fmt={fmt} {rows}x{K} group={group}", flush=True)
    b = _bits(rows, K, rows + K)
    live = max(rows - 2, 1)
    codes = torch.full((rows, K), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.full((rows, K // group), -3.0, device="cuda")
    x = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    n = dev_i32([live])
    F.fq_ckpt_save(dev_bf16(b), rows, K, n, fmt, group, codes, scale)
    F.fq_ckpt_load(codes, scale, rows, K, n, fmt, group, x)
    torch.cuda.synchronize()
    rc, rs = O.ckpt_save(b, fmt, group)
    c, s = codes.cpu().numpy(), scale.cpu().numpy()
    assert np.array_equal(c[:live], rc[:live])
    assert np.array_equal(s[:live], rs[:live], equal_nan=True)
    got, want = host_bits(x), O.ckpt_load(rc, rs, fmt)
    nan = np.isnan(bf16_vals(want))
    assert np.array_equal(np.isnan(bf16_vals(got))[:live], nan[:live])
    assert np.array_equal(got[:live][~nan[:live]], want[:live][~nan[:live]])
    # rows behind the last are left as they were
    assert np.all(c[live:] == 0xA5) and np.all(s[live:] == -3.0)
    assert np.all(bf16_vals(got[live:]) == 7.0)
    # NULL n_rows: all rows
    F.fq_ckpt_save(dev_bf16(b), rows, K, None, fmt, group, codes, scale)
    F.fq_ckpt_load(codes, scale, rows, K, None, fmt, group, x)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scale.cpu().numpy(), rs, equal_nan=True)


ACTS = [(O.FMT_NONE, 1.0), (O.FMT_NVFP4, 0.004), (O.FMT_FP8, 0.02), (O.FMT_INT8, 0.05)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("afmt,as_", ACTS)
@pytest.mark.parametrize("R,live,Fc,group", [(1, 1, 16, 16), (9, 7, 80, 16), (130, 130, 768, 128),
                                             (33, 32, 512, 512), (5, 0, 48, 16)])
def test_swiglu_forward_equals_the_plain_call_and_save(fmt, afmt, as_, R, live, Fc, group):
    b = _bits(R, 2 * Fc, 5 + R, specials=False)
    h, n = dev_bf16(b), dev_i32([live])
    aq = F.ActQ(afmt, dev_f32([as_]))

    def bufs():
        return [torch.full((R, Fc), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    a1, q1 = bufs()
    a2, q2 = bufs()
    codes = torch.full((R, 2 * Fc), 0xA5, dtype=torch.uint8, device="cuda")
    c2 = codes.clone()
    scale = torch.full((R, 2 * Fc // group), -3.0, device="cuda")
    s2 = scale.clone()
    F.fq_swiglu_actfq(h, R, n, Fc, aq, a1, q1)
    F.fq_swiglu_actfq_ckpt(h, R, n, Fc, aq, fmt, group, a2, q2, codes, scale)
    F.fq_ckpt_save(h, R, 2 * Fc, n, fmt, group, c2, s2)
    for x, y in ((a1, a2), (q1, q2), (codes, c2), (scale, s2)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    q3 = torch.full((R, Fc), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fq_swiglu_actfq_ckpt(h, R, n, Fc, aq, fmt, group, None, q3, codes, scale)
    assert torch.equal(q1.view(torch.int16), q3.view(torch.int16))


@pytest.mark.parametrize("afmt,as_", ACTS)
def test_swiglu_backward_bitwise_where_the_saved_values_are_bf16(afmt, as_):
    """INT8 codes times a power of two are bf16 values: the plain backward and
    forward on the loaded tensor give the same bits."""
    R, Fc, group = 70, 160, 32
    rng = np.random.default_rng(11)
    codes = torch.from_numpy(rng.integers(-127, 128, (R, 2 * Fc)).astype(np.int8)).cuda()
    codes = codes.view(torch.uint8)
    scale = dev_f32(2.0 ** rng.integers(-8, -3, (R, 2 * Fc // group)))
    daq, n = dev_bf16(_bits(R, Fc, 1, specials=False)), dev_i32([R - 3])
    aq = F.ActQ(afmt, dev_f32([as_]))
    h = torch.zeros(R, 2 * Fc, dtype=torch.bfloat16, device="cuda")
    F.fq_ckpt_load(codes, scale, R, 2 * Fc, None, O.FMT_INT8, group, h)
    learn = afmt in (O.FMT_FP8, O.FMT_INT8)
    ws = torch.empty(F.fq_workspace_bytes(F.FQ_OP_ACT_SCALE_GRAD, (1, R, Fc), 0, 0),
                     dtype=torch.uint8, device="cuda")
    new = lambda c: torch.full((R, c), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ds = [torch.full((1,), 5.0, device="cuda") if learn else None for _ in range(2)]
    dh1, dh2, q1, q2 = new(2 * Fc), new(2 * Fc), new(Fc), new(Fc)
    F.fq_swiglu_bwd(daq, h, R, n, Fc, aq, dh1, ds[0], ws)
    F.fq_swiglu_actfq(h, R, n, Fc, aq, None, q1)
    F.fq_swiglu_bwd_ckpt(daq, codes, scale, R, n, Fc, O.FMT_INT8, group, aq, dh2, q2, ds[1], ws)
    assert torch.equal(dh1.view(torch.int16), dh2.view(torch.int16))
    assert torch.equal(q1.view(torch.int16), q2.view(torch.int16))
    if learn:
        assert torch.equal(ds[0], ds[1]) and float(ds[0]) != 5.0
    dh3 = new(2 * Fc)
    F.fq_swiglu_bwd_ckpt(daq, codes, scale, R, n, Fc, O.FMT_INT8, group, aq, dh3)
    assert torch.equal(dh1.view(torch.int16), dh3.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("afmt,as_", ACTS)
@pytest.mark.parametrize("R,Fc,group", [(1, 16, 16), (40, 272, 16), (67, 768, 256)])
def test_swiglu_backward_against_float64(fmt, afmt, as_, R, Fc, group):
    """dh and dS_a of the saved values. Where A sits so near a bf16 rounding
    border that fp32 may round it either way, its mask and factor are open and
    the element is left out of the comparison of dh (a mask bit only where it
    differs) and given its whole term in dS_a's tolerance."""
    print(f"[ckpt] bwd fmt={fmt} afmt={afmt} R={R} F={Fc}", flush=True)
    b = _bits(R, 2 * Fc, 21 + R, specials=False)
    daq_b = _bits(R, Fc, 22 + R, specials=False)
    codes, scale = O.ckpt_save(b, fmt, group)
    h = O.ckpt_values(codes, scale, fmt)
    g, u, s, a = O.swiglu_from_values(h)
    # sigmoid on the hardware: exp(-g) carries |g| log2(e) 2^-24 from its
    # argument and a few ulp; A two more products
    rel = (np.abs(g) + 8) * 2.0 ** -23
    lo, hi = O.f64_to_bf16(a * (1 - rel)), O.f64_to_bf16(a * (1 + rel))
    open_ = lo != hi
    f_lo, f_hi = O.fq_act(lo, afmt, as_), O.fq_act(hi, afmt, as_)
    if afmt == O.FMT_NVFP4:                    # an open element opens its block
        blk = open_.reshape(R, -1, 16).any(-1)
        open_ = np.repeat(blk, 16, axis=1)
    assert open_.mean() < 0.2
    aq = F.ActQ(afmt, dev_f32([as_]))
    learn = afmt in (O.FMT_FP8, O.FMT_INT8)
    dh = torch.empty(R, 2 * Fc, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(R, Fc, dtype=torch.bfloat16, device="cuda")
    ds = torch.empty(1, device="cuda") if learn else None
    ws = torch.empty(F.fq_workspace_bytes(F.FQ_OP_ACT_SCALE_GRAD, (1, R, Fc), 0, 0),
                     dtype=torch.uint8, device="cuda")
    F.fq_swiglu_bwd_ckpt(dev_bf16(daq_b), torch.from_numpy(codes).cuda(), dev_f32(scale), R,
                         dev_i32([R]), Fc, fmt, group, aq, dh, q, ds, ws)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(q)[~open_], f_lo.bits[~open_])
    d = bf16_vals(daq_b)
    m = f_lo.mask
    ref = O.swiglu_bwd_values(d * m, h)
    got = bf16_vals(host_bits(dh))
    # fp32: six products, 1 + g (1 - s), whose terms may cancel and where s's
    # error enters times g, then half a bf16 step
    mag = np.concatenate([np.abs(d * u * s) * (1 + np.abs(g)), np.abs(d * g * s)], 1)
    tol = 2.0 ** -8 * np.abs(ref) + np.tile(rel + 8 * 2.0 ** -24, 2) * mag * 1.01 + 2.0 ** -133
    skip = np.tile(open_ & (f_lo.mask != f_hi.mask) if afmt != O.FMT_NVFP4 else open_, 2)
    assert np.all((np.abs(got - ref) <= tol) | skip)
    if learn:
        t_lo, t_hi = d * f_lo.dv_ds, d * f_hi.dv_ds
        # the two candidate terms of an open element, plus the sum's own rounding
        slack = np.abs(t_lo - t_hi).sum() + ACT_DSCALE_TOL * np.abs(t_lo).sum()
        assert abs(float(ds) - t_lo.sum()) <= slack


def test_infinite_gate_reaches_the_gradient():
    """A saved group that held an infinity gives NaN gradients, its neighbours none."""
    b = _bits(4, 128, 9, specials=False)
    b[1, 5] = 0x7F80
    h, n = dev_bf16(b), dev_i32([4])
    codes = torch.empty(4, 128, dtype=torch.uint8, device="cuda")
    scale = torch.empty(4, 8, device="cuda")
    q = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")
    dh = torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    F.fq_swiglu_actfq_ckpt(h, 4, n, 64, None, O.FMT_INT8, 16, None, q, codes, scale)
    F.fq_swiglu_bwd_ckpt(dev_bf16(_bits(4, 64, 8)), codes, scale, 4, n, 64, O.FMT_INT8, 16, None, dh)
    bad = torch.isnan(dh.float()).cpu().numpy()
    want = np.zeros((4, 128), bool)
    want[1, 0:16] = want[1, 64:80] = True
    assert np.array_equal(bad, want)


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 elements (byte offsets beyond 32 bits): the
    first and last rows, and the count of saved bytes in between."""
    K, group = 8192, 512
    rows = (1 << 31) // K + 9
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[0], x[-1] = 3.0, -5.0
    codes = torch.full((rows, K), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, K // group, device="cuda")
    F.fq_ckpt_save(x, rows, K, None, O.FMT_INT8, group, codes, scale)
    assert torch.all(codes[0] == 127) and torch.all(codes[-1] == 0x81)
    assert not codes[1:-1].any()
    y = torch.full_like(x, 7.0)
    F.fq_ckpt_load(codes, scale, rows, K, None, O.FMT_INT8, group, y)
    assert torch.equal(y, x)


def test_no_rows_launch_nothing():
    for call in (lambda: F.fq_ckpt_save(None, 0, 64, None, O.FMT_INT8, 16, None, None),
                 lambda: F.fq_ckpt_load(None, None, 0, 64, None, O.FMT_FP8, 16, None),
                 lambda: F.fq_swiglu_actfq_ckpt(None, 0, dev_i32([0]), 64, None, O.FMT_INT8, 16,
                                                None, None, None, None),
                 lambda: F.fq_swiglu_bwd_ckpt(None, None, None, 0, dev_i32([0]), 64, O.FMT_INT8, 16,
                                              None, None)):
        call()
    ds = torch.full((1,), 5.0, device="cuda")
    F.fq_swiglu_bwd_ckpt(None, None, None, 0, dev_i32([0]), 64, O.FMT_INT8, 16,
                         F.ActQ(O.FMT_FP8, dev_f32([0.5])), None, None, ds,
                         torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert float(ds) == 0.0


def test_other_stream_and_graph_replay():
    R, Fc, group = 300, 256, 64
    h, daq = dev_bf16(_bits(R, 2 * Fc, 2)), dev_bf16(_bits(R, Fc, 3))
    n, aq = dev_i32([R - 1]), F.ActQ(O.FMT_FP8, dev_f32([0.02]))
    ws = torch.empty(F.fq_workspace_bytes(F.FQ_OP_ACT_SCALE_GRAD, (1, R, Fc), 0, 0),
                     dtype=torch.uint8, device="cuda")
    out = [torch.zeros(R, Fc, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(R, 2 * Fc, dtype=torch.uint8, device="cuda"),
           torch.zeros(R, 2 * Fc // group, device="cuda"),
           torch.zeros(R, 2 * Fc, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(R, Fc, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")]

    def step():
        F.fq_swiglu_actfq_ckpt(h, R, n, Fc, aq, O.FMT_FP8, group, None, out[0], out[1], out[2])
        F.fq_swiglu_bwd_ckpt(daq, out[1], out[2], R, n, Fc, O.FMT_FP8, group, aq, out[3], out[4],
                             out[5], ws)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    for t in out:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(out, want))
        step()
        torch.cuda.synchronize()
