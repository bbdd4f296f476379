"""The recomputing layer, the layer over int8 codes and the block around it, run
together as a user runs them."""
import numpy as np
import pytest
import torch

import oracle as O
from block_case import a_bracket
from helpers import bf16_vals, check_gemm_tol, dev_bf16, dev_f32, dev_i32, host_bits
from test_gpu_layer_ckpt import FORMATS, bits, make, same
import workloads as W

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None


@pytest.mark.parametrize("name,wfmt,afmt,group", FORMATS)
def test_recomputing_step(name, wfmt, afmt, group):
    """The parts equal the calls, bit for bit. Without an activation format out and dX are
    the layer's that keeps h within the grouped GEMM's tolerance; with one they need not be:
    that layer rounds h to bf16 (2^-8 of A in the end), so an A within 2^-8 of a border of
    the quantizer may take the next value, for E2M1 a third of it away or more, and so does
    one A in a few dozen."""
    plain, x, ids, p, dout = make(wfmt, afmt, group)
    layer, *_ = make(wfmt, afmt, group, recompute=True)
    T, R, ws = x.shape[0], plain.R_max, plain.ws
    outs = []
    for m in (plain, layer):
        m.quantize_weights()
        m.forward(x, ids, p)
        outs.append(host_bits(m.out))
    if afmt == O.FMT_NONE:
        check_gemm_tol(outs[1], outs[0], "out")
    xq = torch.empty_like(x)
    F.fq_actfq(x, T, layer.H, layer.aq1, xq)
    aq = torch.empty_like(layer.aq)
    F.fq_grouped_gated_fwd(xq, T, layer.perm, layer.topk, R, layer.seg, layer.shape_gu, layer.wfq_gu,
                           layer.aq2, aq, ws)
    assert same(bits(aq), bits(layer.aq))
    o, out = torch.empty_like(layer.o), torch.empty_like(layer.out)
    F.fq_grouped_gemm_fwd(aq, R, layer.seg, layer.shape_d, None, layer.wfq_d, layer.q_d, None, o, ws)
    F.fq_moe_combine(o, p, layer.row_of[:T], T, layer.topk, layer.H, out)
    assert same(bits(out), bits(layer.out))
    dx0, *_ = plain.backward(x, p, dout)
    dx, ds_gu, ds_d = layer.backward(x, p, dout)
    if afmt == O.FMT_NONE:
        check_gemm_tol(host_bits(dx), host_bits(dx0), "dx")
    got = bits(dx, ds_gu, ds_d)
    dh, aq2 = torch.empty_like(layer.dh), torch.empty_like(layer.aq)
    F.fq_grouped_gated_bwd(layer.daq, xq, T, layer.perm, layer.topk, R, layer.seg, layer.shape_gu,
                           layer.wfq_gu, layer.aq2, dh, aq2, ws)
    assert same(bits(aq2), bits(aq)) and same(bits(dh), bits(layer.dh))
    z = lambda q: torch.empty_like(q.scale) if wfmt == O.FMT_INT4 else None  # noqa: E731
    g2, d2 = torch.empty_like(ds_gu), torch.empty_like(ds_d)
    F.fq_grouped_gemm_bwd_scale(layer.do, aq, R, layer.seg, layer.shape_d, layer.w_d, layer.wfq_d, layer.q_d,
                                None, None, d2, z(layer.q_d), ws)
    F.fq_grouped_gemm_wgrad_tokens(dh, xq, T, layer.perm, layer.topk, R, layer.seg, layer.shape_gu, layer.w_gu,
                                   layer.q_gu, g2, z(layer.q_gu), ws)
    dxq, dx2 = torch.empty_like(layer.dxq), torch.empty_like(layer.dx)
    F.fq_grouped_gemm_bwd_scale(dh, None, R, layer.seg, layer.shape_gu, layer.w_gu, layer.wfq_gu, layer.q_gu,
                                None, dxq, None, None, ws)
    F.fq_moe_unpermute_reduce(dxq, layer.row_of[:T], x, T, layer.topk, layer.H, layer.aq1, dx2, None, None)
    assert same(bits(dx2, g2, d2), got)


def test_recomputing_layers_share_their_buffers():
    """Two layers in a row over one set of buffers: the bits of layers with their own;
    an input that the buffers no longer hold is refused."""
    def chain(shared):
        l1, x, ids, p, dout = make(O.FMT_FP8, O.FMT_FP8, None, seed=5, recompute=True)
        l2, _, ids2, p2, _ = make(O.FMT_FP8, O.FMT_FP8, None, seed=6, recompute=True,
                                  **({"scratch_of": l1} if shared else {}))
        out = []
        for step in range(2):
            for m in (l1, l2):
                m.quantize_weights()
            y = l1.forward(x, ids, p).clone()
            z = l2.forward(y, ids2, p2)
            out += bits(z)
            if shared:
                with pytest.raises(ValueError):
                    l2.backward(z, p2, dout)
            d2, g2, s2 = l2.backward(y, p2, dout)
            d2 = d2.clone()
            d1, g1, s1 = l1.backward(x, p, d2)
            out += bits(d1, g2, s2, g1, s1)
        return out

    assert same(chain(False), chain(True))


def test_recompute_refusals():
    for kw in (dict(ckpt=(O.FMT_INT8, 64)), dict(learn_act_scales=True)):
        with pytest.raises(ValueError):
            make(O.FMT_FP8, O.FMT_FP8, None, recompute=True, **kw)
    ck, *_ = make(O.FMT_FP8, O.FMT_FP8, None, ckpt=(O.FMT_INT8, 64))
    with pytest.raises(ValueError):
        make(O.FMT_FP8, O.FMT_FP8, None, recompute=True, scratch_of=ck)
    layer, x, ids, p, dout = make(O.FMT_FP8, O.FMT_FP8, None, recompute=True)
    layer.quantize_weights()
    with pytest.raises(ValueError):
        layer.forward(x, ids, p, keep_a=True)
    layer.forward(x, ids, p)
    with pytest.raises(ValueError):
        layer.backward(None, p, dout)


def int8_layer(group=None, local=False, T=150):
    case = W.moe_case(T=T, fmt="int8", E_global=8, H=272, F=144, topk=3, seed=11,
                      expert_begin=2 if local else 0, E_local=3 if local else None)
    layer = F.MoEFakeQuantLayer(dev_bf16(case.w_gu), dev_bf16(case.w_d), O.FMT_INT8, O.FMT_INT8, T, 3,
                                2 if local else 0, group)
    x, ids, p = dev_bf16(case.x), dev_i32(case.expert_ids), dev_f32(case.probs)
    layer.init_weight_scales()
    layer.export()
    return layer, x, ids, p


@pytest.mark.parametrize("group", [None, -1])
@pytest.mark.parametrize("local", [False, True])
@pytest.mark.parametrize("T", [1, 7, 150])
def test_layer_over_int8_codes(group, local, T):
    """Stage by stage, each fed the stage before it."""
    print(f"[layer int8] group={group} local={local} T={T}", flush=True)
    layer, x, ids, p = int8_layer(group, local)
    gu, d = layer.stored
    out = layer.forward_int8(x[:T], ids[:T], p[:T])
    b = {k: v.cpu() for k, v in layer.i8.items() if k != "ws"}
    n = lambda t: t.cpu().numpy()  # noqa: E731
    perm, row_of, seg = O.moe_permute(n(ids[:T]), layer.expert_begin, layer.E)
    R = int(seg[-1])
    assert np.array_equal(b["seg"].numpy(), seg) and np.array_equal(b["perm"].numpy()[:R], perm[:R])
    xc, sx = O.quantize_tokens(host_bits(x[:T]))
    assert np.array_equal(b["x_codes"].numpy()[:T], xc) and np.array_equal(b["x_scale"].numpy()[:T], sx)
    shaped = lambda st, shape: n(st.codes).reshape(shape)  # noqa: E731
    scales = lambda st: n(st.scale).reshape(layer.E, -1).squeeze(1) if group == -1 else n(st.scale)[..., 0]  # noqa: E731
    lo, hi, _ = a_bracket(O.int8_sums(xc, sx, perm, 3, seg, shaped(gu, layer.shape_gu), scales(gu)))
    a = host_bits(b["a"])[:R]
    assert np.all((bf16_vals(a) >= bf16_vals(lo)) & (bf16_vals(a) <= bf16_vals(hi)))
    ac, sa = O.quantize_tokens(a)
    assert np.array_equal(b["a_codes"].numpy()[:R], ac) and np.array_equal(b["a_scale"].numpy()[:R], sa)
    o = O.gemm_int8(ac, sa, None, 1, seg, shaped(d, layer.shape_d), scales(d))
    assert np.array_equal(host_bits(b["o"])[:R], o)
    ref = bf16_vals(O.combine(o, n(p[:T]), row_of))
    # three fp32 products and sums, then half a bf16 step on either side of the reference
    mag = bf16_vals(O.combine(o & 0x7FFF, np.abs(n(p[:T])), row_of))
    assert np.all(np.abs(bf16_vals(host_bits(out)) - ref) <= 2.0 ** -8 * np.abs(ref) * 2 + 2.0 ** -20 * mag)


def test_layer_over_int8_codes_refusals():
    layer, x, ids, p = int8_layer()
    for bad in ((x[:4], ids[:3], p[:4]), (x[:4], ids[:4], p[:4].half()), (x[:4, :256], ids[:4], p[:4]),
                (x[:4].float(), ids[:4], p[:4]), (x.repeat(2, 1), ids.repeat(2, 1), p.repeat(2, 1))):
        with pytest.raises(ValueError):
            layer.forward_int8(*bad)
    other, x, ids, p, _ = make(O.FMT_FP8, O.FMT_FP8, None)
    with pytest.raises(ValueError):
        other.forward_int8(x, ids, p)                       # not exported
    other.export()
    with pytest.raises(ValueError):
        other.forward_int8(x, ids, p)                       # not int8
    grouped, x, ids, p, _ = make(O.FMT_INT8, O.FMT_INT8, 64)
    grouped.export()
    with pytest.raises(ValueError):
        grouped.forward_int8(x, ids, p)                     # groups inside a row


def block_of(layer, post=True, **kw):
    rng = np.random.default_rng(3)
    w = lambda: dev_bf16(O.f32_to_bf16((1 + 0.2 * rng.standard_normal(layer.H)).astype(np.float32)))  # noqa: E731
    return F.MoEFakeQuantBlock(layer, w(), w() if post else None, alpha=0.6, **kw)


@pytest.mark.parametrize("post,gated", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("mode", [dict(), dict(recompute=True), dict(ckpt=(O.FMT_INT8, 64))])
def test_block_step(post, gated, mode):
    """The block's step is the norms' calls around the layer's step."""
    layer, x, ids, p, dy = make(O.FMT_FP8, O.FMT_FP8, None, **mode)
    ref, *_ = make(O.FMT_FP8, O.FMT_FP8, None, **mode)
    T, H, eps = x.shape[0], layer.H, 1e-6
    blk = block_of(layer, post, learn_norms=True)
    gate = torch.sigmoid(torch.randn(T, device="cuda", generator=torch.Generator("cuda").manual_seed(1))) \
        if gated else None
    layer.quantize_weights()
    y = blk.forward(x, ids, p, gate)
    got = bits(y)
    dx, ds_gu, ds_d = blk.backward(p, dy)
    got += bits(dx, ds_gu, ds_d, blk.dw_pre)
    if gated:
        got += bits(blk.dgate[:T])
    if post:
        got += bits(blk.dw_post)
    # by the calls
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    n, y2, db, dx2 = e(T, H), e(T, H), e(T, H), e(T, H)
    dg = e(T, t=torch.float32) if gated else None
    dwo, dwp = (e(H, t=torch.float32) if post else None), e(H, t=torch.float32)
    ref.quantize_weights()
    F.fq_norm_residual_fwd(x, None, None, 1.0, None, blk.w_pre, eps, T, H, None, n)
    b = ref.forward(n, ids, p).clone()
    F.fq_norm_residual_fwd(x, b, gate, 0.6, blk.w_post, None, eps, T, H, y2)
    F.fq_norm_residual_bwd(dy, None, None, b, gate, 0.6, blk.w_post, None, eps, T, H, None, db, dg, dwo, None,
                           blk.ws)
    dn, g2, d2 = ref.backward(n, p, db)
    F.fq_norm_residual_bwd(dy, dn, x, None, None, 1.0, None, blk.w_pre, eps, T, H, dx2, None, None, None, dwp,
                           blk.ws)
    want = bits(y2, dx2, g2, d2, dwp) + (bits(dg) if gated else []) + (bits(dwo) if post else [])
    assert same(got, want)
    # and y against float64 from b
    v = lambda t: None if t is None else bf16_vals(host_bits(t))  # noqa: E731
    f = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    ry, _ = O.norm_residual(v(x), v(b), f(gate), float(np.float32(0.6)), v(blk.w_post), None,
                            float(np.float32(eps)))
    k = (H / 2 + 12) * 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(ry) + 1.01 * (k * np.abs(ry - v(x)) + 2.0 ** -23 * np.abs(ry))
    assert np.all(np.abs(bf16_vals(host_bits(y2)) - ry) <= tol)


def test_block_over_int8_codes_and_replays():
    """The served block: the norm's codes go straight into the products. Captured and
    replayed over new tokens, with a training step of another block between."""
    layer, x, ids, p = int8_layer()
    T = x.shape[0]
    blk = block_of(layer)
    gate = torch.rand(T, device="cuda")
    y = blk.forward_int8(x, ids, p, gate)
    codes = torch.empty(T, layer.H, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, device="cuda")
    F.fq_norm_residual_fwd(x, None, None, 1.0, None, blk.w_pre, 1e-6, T, layer.H, None, None, codes, s)
    b = layer.forward_int8_codes(codes, s, T, ids, p)
    y2 = torch.empty_like(y)
    F.fq_norm_residual_fwd(x, b, gate, 0.6, blk.w_post, None, 1e-6, T, layer.H, y2)
    assert same(bits(y), bits(y2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk.forward_int8(x, ids, p, gate)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = blk.forward_int8(x, ids, p, gate)
    train, tx, tids, tp, tdy = make(O.FMT_FP8, O.FMT_FP8, None, recompute=True)
    tb = block_of(train, learn_norms=True)

    def step():
        train.quantize_weights()
        tb.forward(tx, tids, tp)
        return (*tb.backward(tp, tdy), tb.dw_pre, tb.dw_post)

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gt = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gt):
        touts = step()
    first = None
    for rep in range(3):
        x.copy_(torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(rep)).bfloat16())
        got = bits(*step())
        first = first or got
        assert same(got, first)
        for t in touts:
            t.zero_()
        gt.replay()
        assert same(bits(*touts), first)
        out.zero_()
        g.replay()
        got = bits(out)
        assert same(got, bits(blk.forward_int8(x, ids, p, gate)))


def test_block_refusals():
    layer, x, ids, p, dy = make(O.FMT_FP8, O.FMT_FP8, None)
    with pytest.raises(ValueError):
        F.MoEFakeQuantBlock(layer, torch.ones(layer.H, device="cuda"))
    blk = block_of(layer)
    with pytest.raises(ValueError):
        blk.backward(p, dy)
    with pytest.raises(ValueError):
        blk.forward(layer.out, ids, p)
    for bad in ((x[:, :64], None), (x.float(), None), (torch.cat((x, x)), None), (x, torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            blk.forward(bad[0], ids, p, bad[1])
    blk.forward(x, ids, p)
    with pytest.raises(ValueError):
        blk.backward(p, dy[:4])


def test_another_device_and_layouts_are_refused():
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    for bad in (x.cpu(), x.t(), torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            F.fq_norm_residual_fwd(bad, None, None, 1.0, None, w, 1e-6, 4, 32, None, torch.empty_like(x))
    with pytest.raises(ValueError):
        F.fq_norm_residual_fwd(x.float(), None, None, 1.0, None, w, 1e-6, 4, 32, None, torch.empty_like(x))
    with pytest.raises(TypeError):
        F.fq_norm_residual_fwd(x.data_ptr(), None, None, 1.0, None, w, 1e-6, 4, 32, None, torch.empty_like(x))
    with pytest.raises(F.FQError):
        F.fq_norm_residual_fwd(x, None, None, 1.0, None, w, 0.0, 4, 32, None, torch.empty_like(x))
    with pytest.raises(OverflowError):
        F.fq_norm_residual_fwd(x, None, None, 1.0, None, w, 1e-6, 1 << 40, 32, None, torch.empty_like(x))


def test_block_refuses_inputs_that_its_own_calls_overwrite():
    """A block's or its layer's own buffers: as x of a training step (kept until the
    backward), as dy, and the int8 layer's output as x of the int8 form."""
    layer, x, ids, p, dy = make(O.FMT_INT8, O.FMT_INT8, None)
    T = x.shape[0]
    blk = block_of(layer)
    layer.quantize_weights()
    y = blk.forward(x, ids, p)
    for bad in (y, blk.dx[:T], layer.out[:T]):
        with pytest.raises(ValueError):
            blk.forward(bad, ids, p)
    for bad in (blk.db[:T], layer.dx[:T]):
        with pytest.raises(ValueError):
            blk.backward(p, bad)
    first = bits(blk.backward(p, dy)[0])
    blk.dx[:T].copy_(dy)  # the block's own dx may be dy
    assert same(bits(blk.backward(p, blk.dx[:T])[0]), first)
    layer.export()
    z = layer.forward_int8(x, ids, p)
    with pytest.raises(ValueError):
        blk.forward_int8(z, ids, p)
    want = bits(blk.forward_int8(x, ids, p))
    blk.y[:T].copy_(x)  # in place on the block's own y
    assert same(bits(blk.forward_int8(blk.y[:T], ids, p)), want)


@pytest.mark.parametrize("post,gated", [(True, True), (False, False)])
@pytest.mark.parametrize("mode", [dict(), dict(recompute=True), dict(ckpt=(O.FMT_INT8, 64))])
def test_block_without_tokens(post, gated, mode):
    """A rank that no token reaches: empty results, and weights' gradients of zero."""
    layer, x, ids, p, dy = make(O.FMT_INT8, O.FMT_INT8, None, **mode)
    blk = block_of(layer, post, learn_norms=True)
    gate = torch.ones(0, device="cuda") if gated else None
    layer.quantize_weights()
    layer.export()
    blk.dw_pre.fill_(7.0)
    assert blk.forward(x[:0], ids[:0], p[:0], gate).shape == (0, layer.H)
    dx, ds_gu, ds_d = blk.backward(p[:0], dy[:0])
    assert dx.shape == (0, layer.H) and not ds_gu.any() and not ds_d.any() and not blk.dw_pre.any()
    assert not post or not blk.dw_post.any()
    assert blk.forward_int8(x[:0], ids[:0], p[:0], gate).shape == (0, layer.H)


def test_block_refuses_other_rows_of_the_buffers_it_writes():
    """x within y, or dy within dx, at another row: written in place, a row would overwrite
    one that is still to be read. The same for the int8 layer's inner buffers as x."""
    layer, x, ids, p, dy = make(O.FMT_INT8, O.FMT_INT8, None)
    T = x.shape[0]
    blk = block_of(layer)
    layer.quantize_weights()
    layer.export()
    blk.forward_int8(x, ids, p)
    n = T - 3
    for bad in (blk.y[3:T], layer.i8["o"][:n], layer.i8["o"][5:5 + n]):
        with pytest.raises(ValueError):
            blk.forward_int8(bad, ids[:n], p[:n])
    blk.forward(x[:n], ids[:n], p[:n])
    with pytest.raises(ValueError):
        blk.backward(p[:n], blk.dx[3:T])
    # fewer rows from the first one on are in place row by row
    blk.dx[:n].copy_(dy[:n])
    got = bits(blk.backward(p[:n], blk.dx[:n])[0])
    assert same(got, bits(blk.backward(p[:n], dy[:n])[0]))


def test_block_refuses_its_gate_gradient_as_the_gate():
    """The gate is kept by reference: the first backward would overwrite it."""
    layer, x, ids, p, dy = make(O.FMT_FP8, O.FMT_FP8, None)
    blk = block_of(layer)
    layer.quantize_weights()
    blk.dgate.fill_(0.5)
    T = x.shape[0]
    with pytest.raises(ValueError):
        blk.forward(x, ids, p, blk.dgate[:T])
    blk.forward(x, ids, p, blk.dgate[:T].clone())
    first = bits(blk.backward(p, dy)[0])
    assert same(bits(blk.backward(p, dy)[0]), first)
