"""GPU parity of the token int8 codes, the int8 products and the gated block
through the C ABI, against float64 (int8: bit for bit)."""
import numpy as np
import pytest
import torch

import oracle as O
from block_case import a_bracket, codes, exact_bits, normal_bits, route
from helpers import bf16_vals, dev_bf16, dev_f32, dev_i32, host_bits
from test_gpu_graph import _capture

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

FILL = 7.0


def dev_u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def out_bf16(*shape):
    return torch.full(shape, FILL, dtype=torch.bfloat16, device="cuda")


def workspace(op, shape, R):
    return torch.empty(max(256, F.fq_workspace_bytes(op, shape, R, 0)), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ token codes --
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 4096), (5, 48), (130, 512), (33, 1040), (7, 2064),
                                    (3, 8208), (2, 16400), (2, 33008)])
def test_token_codes_bitexact(rows, K):
    print(f"[tokens] {rows}x{K}", flush=True)
    rng = np.random.default_rng(rows + K)
    b = normal_bits(rng, rows, K)
    if rows > 2:
        b[0] = 0x8000                                        # negative zeros: scale 1
        b[1, K - 1] = 0x7F80                                 # +inf in the last column
        b[2] = rng.integers(0, 8, K)                         # subnormals
    live = max(1, rows - 1)
    c, s = torch.full((rows, K), 0xA5, dtype=torch.uint8, device="cuda"), dev_f32(np.full(rows, -3.0))
    F.fq_quantize_tokens(dev_bf16(b), rows, K, dev_i32([live]), c, s)
    rc, rs = O.quantize_tokens(b)
    assert np.array_equal(c.cpu().numpy()[:live], rc[:live])
    assert np.array_equal(s.cpu().numpy()[:live], rs[:live], equal_nan=True)
    assert np.all(c.cpu().numpy()[live:] == 0xA5) and np.all(s.cpu().numpy()[live:] == -3.0)
    F.fq_quantize_tokens(dev_bf16(b), rows, K, None, c, s)
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


# ---------------------------------------------------------- int8 products --
# (E, T, topk, N, K, spare rows, skewed routing)
INT8 = [(1, 1, 1, 16, 16, 0, False), (1, 1, 1, 512, 4096, 0, False), (1, 16, 1, 272, 80, 0, False),
        (1, 17, 1, 48, 1040, 3, False), (4, 9, 3, 64, 48, 2, False), (5, 50, 2, 96, 272, 7, True),
        (3, 300, 1, 1040, 368, 11, True), (2, 257, 2, 512, 128, 0, False), (1, 600, 1, 256, 640, 1, False),
        (7, 150, 4, 304, 400, 40, True), (130, 40, 2, 32, 64, 5, False), (1, 33, 1, 4096, 144, 0, False),
        # enough tiles of 256, and of 128 (more than CUs, and fewer), to be taken
        (64, 1300, 4, 1056, 144, 60, True), (64, 1300, 4, 1056, 656, 0, False),
        (16, 700, 3, 1056, 272, 9, True), (8, 800, 3, 1056, 400, 5, False)]


@pytest.mark.parametrize("E,T,topk,N,K,spare,skew", INT8)
@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("tensor", [False, True])
def test_int8_product_bitexact(E, T, topk, N, K, spare, skew, routed, tensor):
    print(f"[int8] E={E} T={T} topk={topk} N={N} K={K} routed={routed} tensor={tensor}", flush=True)
    rng = np.random.default_rng(E * T + N + K)
    perm, seg = route(rng, T, topk, E, skew, spare)
    R, live = T * topk, int(seg[-1])
    rows = T if routed else R
    xc, wc = codes(rng, rows, K), codes(rng, E, N, K)
    sx = (rng.random(rows) + 0.01).astype(np.float32)
    sw = (rng.random(E if tensor else (E, N)) * 1e-2).astype(np.float32)
    p = perm if routed else None
    want = O.gemm_int8(xc, sx, p, topk, seg, wc, sw)
    st = F.StoredW(F.FMT_INT8, F.FQ_GROUP_TENSOR if tensor else K, dev_u8(wc), dev_f32(sw))
    y = out_bf16(R, N)
    F.fq_grouped_gemm_int8(dev_u8(xc), dev_f32(sx), rows, dev_i32(perm) if routed else None, topk, R,
                           dev_i32(seg), (E, N, K), st, y, workspace(F.FQ_OP_GEMM_INT8, (E, N, K), R))
    got = host_bits(y)
    assert np.array_equal(got[:live], want)
    assert np.all(bf16_vals(got[live:]) == FILL)


@pytest.mark.parametrize("E,T,topk,N,K,spare,skew", [c for c in INT8 if c[3] % 32 == 0])
def test_int8_gated_product(E, T, topk, N, K, spare, skew):
    print(f"[int8 gated] E={E} T={T} topk={topk} 2F={N} K={K}", flush=True)
    rng = np.random.default_rng(E * T + N + K + 1)
    perm, seg = route(rng, T, topk, E, skew, spare)
    R, live = T * topk, int(seg[-1])
    xc, wc = codes(rng, T, K), codes(rng, E, N, K)
    sx = ((rng.random(T) + 0.1) * 2e-3).astype(np.float32)
    sw = ((rng.random((E, N)) + 0.1) * 1e-2 / np.sqrt(K)).astype(np.float32)
    # g and u are the exact sums times two fp32 scales, as float64 takes them here
    lo, hi, _ = a_bracket(O.int8_sums(xc, sx, perm, topk, seg, wc, sw))
    st = F.StoredW(F.FMT_INT8, K, dev_u8(wc), dev_f32(sw))
    a = out_bf16(R, N // 2)
    F.fq_grouped_gated_int8(dev_u8(xc), dev_f32(sx), T, dev_i32(perm), topk, R, dev_i32(seg), (E, N, K),
                            st, a, workspace(F.FQ_OP_GATED, (E, N, K), R))
    got = bf16_vals(host_bits(a))
    assert np.all((got[:live] >= bf16_vals(lo)) & (got[:live] <= bf16_vals(hi)))
    assert np.all(got[live:] == FILL)


def test_int8_extremes_of_the_sum():
    """All codes -128: the largest sums that an int32 holds."""
    K, N = 131056, 16
    xc, wc = np.full((1, K), 0x80, np.uint8), np.full((1, N, K), 0x80, np.uint8)
    wc[0, 1] = 0x7F
    st = F.StoredW(F.FMT_INT8, K, dev_u8(wc), dev_f32(np.ones((1, N))))
    y = out_bf16(1, N)
    F.fq_grouped_gemm_int8(dev_u8(xc), dev_f32([1.0]), 1, None, 1, 1, dev_i32([0, 1]), (1, N, K), st, y,
                           workspace(F.FQ_OP_GEMM_INT8, (1, N, K), 1))
    want = O.gemm_int8(xc, [1.0], None, 1, [0, 1], wc, np.ones((1, N), np.float32))
    assert np.array_equal(host_bits(y), want)


def test_int8_a_row_that_is_not_finite_is_nan_and_alone():
    rng = np.random.default_rng(4)
    R, N, K = 40, 64, 96
    b = normal_bits(rng, R, K)
    b[7, 3], b[21, 0] = 0x7FC0, 0xFF80
    wc, seg = codes(rng, 2, N, K), [0, 20, R]
    c, s, y = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(R, device="cuda"), out_bf16(R, N)
    F.fq_quantize_tokens(dev_bf16(b), R, K, None, c, s)
    st = F.StoredW(F.FMT_INT8, K, dev_u8(wc), dev_f32(np.full((2, N), 0.01)))
    F.fq_grouped_gemm_int8(c, s, R, None, 1, R, dev_i32(seg), (2, N, K), st, y,
                           workspace(F.FQ_OP_GEMM_INT8, (2, N, K), R))
    bad = torch.isnan(y.float()).cpu().numpy()
    want = np.zeros((R, N), bool)
    want[[7, 21]] = True
    assert np.array_equal(bad, want)


# ------------------------------------------------------------ gated block --
# (E, T, topk, H, F, spare rows, skewed routing)
GATED = [(1, 1, 1, 16, 16, 0, False), (1, 1, 1, 2048, 256, 0, False), (1, 16, 1, 80, 48, 0, False),
         (1, 19, 1, 272, 144, 2, False), (4, 9, 3, 48, 32, 2, False), (5, 50, 2, 208, 80, 7, True),
         (2, 257, 2, 64, 256, 0, False), (3, 300, 1, 368, 528, 11, True), (1, 600, 1, 128, 128, 1, False),
         (7, 150, 4, 336, 112, 40, True), (130, 40, 2, 32, 16, 5, False), (1, 130, 1, 1040, 768, 0, False),
         # enough tiles of 256, and of 128 (more than CUs, and fewer), to be taken
         (64, 1300, 4, 144, 528, 60, True), (64, 1300, 4, 272, 640, 0, False),
         (16, 700, 3, 272, 528, 9, True), (8, 800, 3, 208, 528, 5, False)]
ACTS = [(O.FMT_NONE, 1.0), (O.FMT_FP8, 0.02), (O.FMT_INT8, 0.05), (O.FMT_NVFP4, 0.01)]


def _scaled(E, T, topk, H, Fc, spare, skew, seed):
    """x, w with g and u of order one, whatever H."""
    rng = np.random.default_rng(seed)
    perm, seg = route(rng, T, topk, E, skew, spare)
    x = exact_bits(rng, T, H)
    w = exact_bits(rng, E, 2 * Fc, H, step=2.0 ** -round(np.log2(H) / 2) / 2)
    return rng, perm, seg, x, w


def _decided(lo, hi):
    return (bf16_vals(lo) == bf16_vals(hi)).reshape(lo.shape[0], -1, 16)


def _check_fq(got, lo, hi, afmt, as_, live, Fc):
    """got [R, F] bits of FQ_a of an A between lo and hi: monotone for the per-tensor
    formats; NVFP4 blocks whose A is decided have to be equal."""
    f_lo = lo if afmt == O.FMT_NONE else O.fq_act(lo, afmt, as_).bits
    f_hi = hi if afmt == O.FMT_NONE else O.fq_act(hi, afmt, as_).bits
    if afmt == O.FMT_NVFP4:
        # an A is undecided with the chance 2 err / (bf16 step) < 2^-8. A zero A is
        # decided, whatever its sign (lo = -0, hi = +0): values, not bits
        same = np.repeat(_decided(lo, hi).all(-1), 16, axis=1)
        assert same.mean() > 0.7
        assert np.array_equal(bf16_vals(got[:live])[same], bf16_vals(f_lo)[same])
    else:
        g = bf16_vals(got[:live])
        assert np.all((g >= bf16_vals(f_lo)) & (g <= bf16_vals(f_hi)))
    assert np.all(bf16_vals(got[live:]) == FILL)


@pytest.mark.parametrize("afmt,as_", ACTS)
@pytest.mark.parametrize("E,T,topk,H,Fc,spare,skew", GATED)
def test_gated_forward(E, T, topk, H, Fc, spare, skew, afmt, as_):
    print(f"[gated] E={E} T={T} topk={topk} H={H} F={Fc} afmt={afmt}", flush=True)
    _, perm, seg, x, w = _scaled(E, T, topk, H, Fc, spare, skew, E * T + H)
    R, live = T * topk, int(seg[-1])
    lo, hi, _ = a_bracket(O.gated_sums(x, perm, topk, seg, w))
    aq = out_bf16(R, Fc)
    F.fq_grouped_gated_fwd(dev_bf16(x), T, dev_i32(perm), topk, R, dev_i32(seg), (E, 2 * Fc, H),
                           dev_bf16(w), F.ActQ(afmt, dev_f32([as_])), aq,
                           workspace(F.FQ_OP_GATED, (E, 2 * Fc, H), R))
    _check_fq(host_bits(aq), lo, hi, afmt, as_, live, Fc)


@pytest.mark.parametrize("afmt,as_", ACTS)
@pytest.mark.parametrize("E,T,topk,H,Fc,spare,skew", GATED)
def test_gated_backward(E, T, topk, H, Fc, spare, skew, afmt, as_):
    print(f"[gated bwd] E={E} T={T} topk={topk} H={H} F={Fc} afmt={afmt}", flush=True)
    rng, perm, seg, x, w = _scaled(E, T, topk, H, Fc, spare, skew, E * T + H + 5)
    R, live = T * topk, int(seg[-1])
    h = O.gated_sums(x, perm, topk, seg, w)
    lo, hi, err = a_bracket(h)
    d_bits = normal_bits(rng, R, Fc)
    args = (dev_bf16(d_bits), dev_bf16(x), T, dev_i32(perm), topk, R, dev_i32(seg), (E, 2 * Fc, H),
            dev_bf16(w), F.ActQ(afmt, dev_f32([as_])))
    ws = workspace(F.FQ_OP_GATED, (E, 2 * Fc, H), R)
    dh, aq, dh2 = out_bf16(R, 2 * Fc), out_bf16(R, Fc), out_bf16(R, 2 * Fc)
    F.fq_grouped_gated_bwd(*args, dh, aq, ws)
    F.fq_grouped_gated_bwd(*args, dh2, None, ws)
    assert torch.equal(dh.view(torch.int16), dh2.view(torch.int16))
    _check_fq(host_bits(aq), lo, hi, afmt, as_, live, Fc)
    d = bf16_vals(d_bits[:live])
    m_lo = 1.0 if afmt == O.FMT_NONE else O.fq_act(lo, afmt, as_).mask
    m_hi = 1.0 if afmt == O.FMT_NONE else O.fq_act(hi, afmt, as_).mask
    skip = np.zeros((live, Fc), bool) | (m_lo != m_hi)
    if afmt == O.FMT_NVFP4:
        skip = np.repeat(~_decided(lo, hi).all(-1), 16, axis=1)
    g, u, s, _ = O.swiglu_from_values(h)
    ref = O.swiglu_bwd_values(d * m_lo, h)
    # six fp32 products, 1 + g (1 - s), whose terms may cancel and where s's error
    # enters times g, then half a bf16 step
    rel = (np.abs(g) + 8) * 2.0 ** -23
    mag = np.concatenate([np.abs(d * u * s) * (1 + np.abs(g)), np.abs(d * g * s)], 1)
    tol = 2.0 ** -8 * np.abs(ref) + np.tile(rel + 8 * 2.0 ** -24, 2) * mag * 1.01 + 2.0 ** -133
    got = bf16_vals(host_bits(dh))
    assert np.all((np.abs(got[:live] - ref) <= tol) | np.tile(skip, 2))
    assert np.all(got[live:] == FILL)


@pytest.mark.parametrize("E,T,topk,H,Fc", [(1, 3, 1, 1024, 64), (3, 200, 2, 528, 272), (1, 520, 1, 256, 384)])
def test_gated_forward_on_normal_inputs(E, T, topk, H, Fc):
    """Sums in any order: each is within (H + 2) 2^-24 of the sum of magnitudes."""
    print(f"[gated normal] E={E} T={T} H={H} F={Fc}", flush=True)
    rng = np.random.default_rng(8)
    perm, seg = route(rng, T, topk, E)
    x, w = normal_bits(rng, T, H), normal_bits(rng, E, 2 * Fc, H, std=H ** -0.5)
    h = O.gated_sums(x, perm, topk, seg, w)
    mags = O.gated_sums(x & 0x7FFF, perm, topk, seg, w & 0x7FFF)
    dh = (H + 2) * 2.0 ** -24 * np.maximum(mags[:, :Fc], mags[:, Fc:])
    lo, hi, _ = a_bracket(h, dh)
    aq = out_bf16(T * topk, Fc)
    F.fq_grouped_gated_fwd(dev_bf16(x), T, dev_i32(perm), topk, T * topk, dev_i32(seg), (E, 2 * Fc, H),
                           dev_bf16(w), None, aq, workspace(F.FQ_OP_GATED, (E, 2 * Fc, H), T * topk))
    _check_fq(host_bits(aq), lo, hi, O.FMT_NONE, 1.0, T * topk, Fc)


@pytest.mark.parametrize("T,H,Fc", [(5, 48, 32), (300, 80, 144), (600, 336, 400), (2500, 144, 1040),
                                    (9000, 144, 2064)])
def test_gated_nan_stays_in_its_row_and_column(T, H, Fc):
    """A NaN in a token, in the token behind the last row's, and in one weight row of
    each expert: the ends of rows inside a tile bring nothing of the neighbours in."""
    rng = np.random.default_rng(9)
    E = 2
    x, w = exact_bits(rng, T, H), exact_bits(rng, E, 2 * Fc, H, step=0.03125)
    x[1], w[0, 2 * Fc - 1], w[1, 0] = 0x7FC0, 0x7FC0, 0x7F80
    perm = np.arange(T, dtype=np.int32)
    seg = np.array([0, T // 2, T - 1], np.int32)
    x[T - 1] = 0x7FC0                                        # a token that no row names
    aq = out_bf16(T, Fc)
    F.fq_grouped_gated_fwd(dev_bf16(x), T, dev_i32(perm), 1, T, dev_i32(seg), (E, 2 * Fc, H), dev_bf16(w),
                           None, aq, workspace(F.FQ_OP_GATED, (E, 2 * Fc, H), T))
    got = aq.float().cpu().numpy()
    bad = ~np.isfinite(got)
    want = np.zeros((T, Fc), bool)
    want[1], want[:T // 2, Fc - 1], want[T // 2:T - 1, 0] = True, True, True
    assert np.array_equal(bad, want)


def test_gated_extreme_gates():
    """Gates far out: silu is 0 (or g itself) there, and its derivative finite."""
    H, Fc = 16, 16
    x = np.zeros((4, H), np.float32)
    x[:, 0], x[:, 1] = [1e4, -1e4, 300.0, -300.0], 1.0
    w = np.zeros((1, 2 * Fc, H), np.float32)
    w[0, :Fc, 0], w[0, Fc:, 1] = 1.0, 2.0
    xb, wb = O.f32_to_bf16(x), O.f32_to_bf16(w)
    args = (dev_bf16(xb), 4, None, 1, 4, dev_i32([0, 4]), (1, 2 * Fc, H), dev_bf16(wb), None)
    aq, dh = out_bf16(4, Fc), out_bf16(4, 2 * Fc)
    ws = workspace(F.FQ_OP_GATED, (1, 2 * Fc, H), 4)
    F.fq_grouped_gated_fwd(*args, aq, ws)
    F.fq_grouped_gated_bwd(torch.ones(4, Fc, dtype=torch.bfloat16, device="cuda"), *args, dh, None, ws)
    g = bf16_vals(xb)[:, 0]
    a = aq.float().cpu().numpy()[:, 0]
    assert a[0] == 2 * g[0] and a[2] == 2 * g[2] and a[1] == 0 and a[3] == 0
    d = dh.float().cpu().numpy()
    assert np.all(d[[0, 2], :Fc] == 2.0) and np.all(d[[1, 3]] == 0.0) and np.all(d[0, Fc:] == g[0])


# --------------------------------------------------------------- together --
def test_no_rows_write_nothing():
    y = out_bf16(4, 32)
    seg0, w = dev_i32([0, 0]), torch.zeros(1, 32, 16, dtype=torch.bfloat16, device="cuda")
    st = F.StoredW(F.FMT_INT8, 16, torch.zeros(1, 32, 16, dtype=torch.uint8, device="cuda"),
                   torch.ones(1, 32, device="cuda"))
    xc, sx = torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), torch.ones(4, device="cuda")
    F.fq_quantize_tokens(None, 0, 16, None, None, None)
    F.fq_quantize_tokens(w[0, :4].contiguous(), 4, 16, dev_i32([0]), xc, sx)
    F.fq_grouped_gemm_int8(None, None, 0, None, 1, 0, seg0, (1, 32, 16), st, None)
    F.fq_grouped_gated_fwd(None, 0, None, 1, 0, seg0, (1, 32, 16), w, None, None)
    F.fq_grouped_gated_bwd(None, None, 0, None, 1, 0, seg0, (1, 32, 16), w, None, None)
    ws = workspace(F.FQ_OP_GEMM_INT8, (1, 32, 16), 4)
    F.fq_grouped_gemm_int8(xc, sx, 4, None, 1, 4, seg0, (1, 32, 16), st, y, ws)      # R_max without a row
    ws = workspace(F.FQ_OP_GATED, (1, 32, 16), 4)
    a = out_bf16(4, 16)
    F.fq_grouped_gated_fwd(w[0, :4].contiguous(), 4, None, 1, 4, seg0, (1, 32, 16), w, None, a, ws)
    F.fq_grouped_gated_int8(xc, sx, 4, None, 1, 4, seg0, (1, 32, 16), st, a, ws)
    F.fq_grouped_gated_bwd(a, w[0, :4].contiguous(), 4, None, 1, 4, seg0, (1, 32, 16), w, None, y, None, ws)
    assert torch.all(y == FILL) and torch.all(a == FILL) and torch.all(sx == 1.0)


@pytest.mark.parametrize("T,H,Fc", [(3, 512, 64), (700, 256, 272), (1500, 256, 1040), (9000, 208, 1040)])
def test_repeats_streams_and_replays_are_bitwise_equal(T, H, Fc):
    """The w8a8 chain and the gated block with its backward: again, on another
    stream with a workspace of its own, and from a captured graph over new inputs."""
    print(f"[blocks graph] T={T} H={H} F={Fc}", flush=True)
    rng = np.random.default_rng(12)
    E, topk = 4, 2
    perm, seg = route(rng, T, topk, E, True, 3 if T > 3 else 1)
    R = T * topk
    x, w = dev_bf16(normal_bits(rng, T, H)), dev_bf16(normal_bits(rng, E, 2 * Fc, H, std=0.05))
    daq = dev_bf16(normal_bits(rng, R, Fc))
    wc, wd = codes(rng, E, 2 * Fc, H), codes(rng, E, H, Fc)
    gu = F.StoredW(F.FMT_INT8, H, dev_u8(wc), dev_f32(rng.random((E, 2 * Fc)) * 1e-3))
    dn = F.StoredW(F.FMT_INT8, Fc, dev_u8(wd), dev_f32(rng.random((E, H)) * 1e-3))
    perm, seg = dev_i32(perm), dev_i32(seg)
    u8 = dict(dtype=torch.uint8, device="cuda")

    def bufs():
        return dict(xc=torch.zeros(T, H, **u8), sx=torch.zeros(T, device="cuda"), a=out_bf16(R, Fc),
                    ac=torch.zeros(R, Fc, **u8), sa=torch.zeros(R, device="cuda"), o=out_bf16(R, H),
                    aq=out_bf16(R, Fc), dh=out_bf16(R, 2 * Fc), aq2=out_bf16(R, Fc),
                    w1=workspace(F.FQ_OP_GATED, (E, 2 * Fc, H), R),
                    w2=workspace(F.FQ_OP_GEMM_INT8, (E, H, Fc), R))

    def step(b):
        F.fq_quantize_tokens(x, T, H, None, b["xc"], b["sx"])
        F.fq_grouped_gated_int8(b["xc"], b["sx"], T, perm, topk, R, seg, (E, 2 * Fc, H), gu, b["a"], b["w1"])
        F.fq_quantize_tokens(b["a"], R, Fc, seg[E:], b["ac"], b["sa"])
        F.fq_grouped_gemm_int8(b["ac"], b["sa"], R, None, 1, R, seg, (E, H, Fc), dn, b["o"], b["w2"])
        F.fq_grouped_gated_fwd(x, T, perm, topk, R, seg, (E, 2 * Fc, H), w, None, b["aq"], b["w1"])
        F.fq_grouped_gated_bwd(daq, x, T, perm, topk, R, seg, (E, 2 * Fc, H), w, None, b["dh"], b["aq2"],
                               b["w1"])

    outs = ("xc", "sx", "a", "ac", "sa", "o", "aq", "dh", "aq2")

    def same(p, q):
        return all(torch.equal(p[k].view(torch.uint8), q[k].view(torch.uint8)) for k in outs)

    one, two = bufs(), bufs()
    step(one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(two)
    step(one)                       # while the other stream works
    torch.cuda.synchronize()
    assert same(one, two)
    assert torch.equal(one["aq"].view(torch.int16), one["aq2"].view(torch.int16))
    cap = bufs()
    g = _capture(lambda: step(cap))
    for rep in range(3):
        x.copy_(dev_bf16(normal_bits(rng, T, H)))
        for k in outs:
            cap[k].zero_() if cap[k].dtype == torch.uint8 else cap[k].fill_(FILL)
        for k in outs:
            one[k].zero_() if one[k].dtype == torch.uint8 else one[k].fill_(FILL)
        g.replay()
        step(one)
        torch.cuda.synchronize()
        assert same(one, cap), f"replay {rep}"


@pytest.mark.parametrize("T", [5, 300, 3000])
def test_direct_rows_do_not_read_topk(T):
    """topk 0 without perm: the bits of topk 1."""
    rng = np.random.default_rng(T)
    H, Fc = 96, 272
    x, w, d = (dev_bf16(normal_bits(rng, *s)) for s in ((T, H), (2, 2 * Fc, H), (T, Fc)))
    xc, sx = dev_u8(codes(rng, T, H)), dev_f32(rng.random(T))
    st = F.StoredW(F.FMT_INT8, H, dev_u8(codes(rng, 2, 2 * Fc, H)), dev_f32(rng.random((2, 2 * Fc))))
    seg, shape = dev_i32([0, T // 3, T]), (2, 2 * Fc, H)

    def run(topk):
        y, a, aq, dh = out_bf16(T, 2 * Fc), out_bf16(T, Fc), out_bf16(T, Fc), out_bf16(T, 2 * Fc)
        F.fq_grouped_gemm_int8(xc, sx, T, None, topk, T, seg, shape, st, y)
        F.fq_grouped_gated_int8(xc, sx, T, None, topk, T, seg, shape, st, a)
        F.fq_grouped_gated_fwd(x, T, None, topk, T, seg, shape, w, None, aq)
        F.fq_grouped_gated_bwd(d, x, T, None, topk, T, seg, shape, w, None, dh)
        return [t.view(torch.int16) for t in (y, a, aq, dh)]

    assert all(torch.equal(p, q) for p, q in zip(run(0), run(1)))


def test_direct_rows_past_4_gib():
    """Direct rows are not bound to 32-bit offsets: the last rows of an x of more than
    4 GiB."""
    K, N = 16384, 16
    R = (1 << 32) // K + 40
    xc = torch.zeros(R, K, dtype=torch.uint8, device="cuda")
    xc[-1], xc[0] = 1, 2
    st = F.StoredW(F.FMT_INT8, K, torch.ones(1, N, K, dtype=torch.uint8, device="cuda"),
                   torch.ones(1, N, device="cuda"))
    y = out_bf16(R, N)
    F.fq_grouped_gemm_int8(xc, torch.ones(R, device="cuda"), R, None, 1, R, dev_i32([0, R]), (1, N, K), st, y,
                           workspace(F.FQ_OP_GEMM_INT8, (1, N, K), R))
    assert torch.all(y[-1] == K) and torch.all(y[0] == 2 * K) and not y[1:-1].any()
