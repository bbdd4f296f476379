"""The MoE layer with 8-bit checkpoints and its few-token form, run together as
a user runs them: training steps that keep only the checkpoints, layers that
share their buffers, the export, and decoding from it."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from helpers import bf16_vals, dev_bf16, dev_f32, dev_i32, host_bits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

FORMATS = [("nvfp4", O.FMT_NVFP4, O.FMT_NVFP4, 16), ("fp8", O.FMT_FP8, O.FMT_FP8, None),
           ("int4", O.FMT_INT4, O.FMT_NONE, 128), ("int8", O.FMT_INT8, O.FMT_INT8, None)]


def make(wfmt, afmt, group, seed=3, T=70, E=6, H=256, Fc=256, topk=3, **kw):
    case = W.moe_case(T=T, fmt="nvfp4", E_global=E, H=H, F=Fc, topk=topk, seed=seed)
    layer = F.MoEFakeQuantLayer(dev_bf16(case.w_gu), dev_bf16(case.w_d), wfmt, afmt, T, topk, 0,
                                group, **kw)
    x, ids = dev_bf16(case.x), dev_i32(case.expert_ids)
    p, dout = dev_f32(case.probs), dev_bf16(case.dout)
    layer.init_weight_scales()
    layer.calibrate(x, ids)
    return layer, x, ids, p, dout


def bits(*ts):
    torch.cuda.synchronize()
    return [t.detach().clone().view(torch.uint8) for t in ts]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name,wfmt,afmt,group", FORMATS)
@pytest.mark.parametrize("ckpt", [(O.FMT_INT8, 64), (O.FMT_FP8, 32)])
def test_checkpointed_step(name, wfmt, afmt, group, ckpt):
    """The forward is the plain layer's, bit for bit; the backward's parts equal
    the calls on what the checkpoint holds (each of which is tested alone)."""
    learn = afmt in (O.FMT_FP8, O.FMT_INT8)
    plain, x, ids, p, dout = make(wfmt, afmt, group, learn_act_scales=learn)
    layer, *_ = make(wfmt, afmt, group, learn_act_scales=learn, ckpt=ckpt)
    for m in (plain, layer):
        m.quantize_weights()
        m.forward(x, ids, p)
    T, R = x.shape[0], plain.R_max
    assert same(bits(plain.out), bits(layer.out))
    dx, ds_gu, ds_d = layer.backward(x, p, dout)
    got = bits(dx, ds_gu, ds_d)
    # what was saved is h
    codes, scale = torch.empty_like(layer.h_codes), torch.empty_like(layer.h_scale)
    F.fq_ckpt_save(plain.h, R, 2 * plain.F, plain.n_rows, *ckpt, codes, scale)
    assert same(bits(codes, scale), bits(layer.h_codes, layer.h_scale))
    # SwiGLU backward, both dScales and dX from it
    dh, aq = torch.empty_like(layer.dh), torch.empty_like(layer.aq)
    dsa = torch.empty(1, device="cuda") if learn else None
    F.fq_swiglu_bwd_ckpt(layer.daq, codes, scale, R, layer.n_rows, layer.F, *ckpt, layer.aq2, dh,
                         aq, dsa, layer.ws)
    d2, g2 = torch.empty_like(ds_d), torch.empty_like(ds_gu)
    z = torch.empty_like(layer.dzp_d) if wfmt == O.FMT_INT4 else None
    zg = torch.empty_like(layer.dzp_gu) if wfmt == O.FMT_INT4 else None
    F.fq_grouped_gemm_bwd_scale(layer.do, aq, R, layer.seg, layer.shape_d, layer.w_d, layer.wfq_d,
                                layer.q_d, None, None, d2, z, layer.ws)
    xq = torch.empty_like(x)
    F.fq_actfq(x, T, layer.H, layer.aq1, xq)
    F.fq_grouped_gemm_wgrad_tokens(dh, xq, T, layer.perm, layer.topk, R, layer.seg, layer.shape_gu,
                                   layer.w_gu, layer.q_gu, g2, zg, layer.ws)
    dxq, dx2 = torch.empty_like(layer.dxq), torch.empty_like(layer.dx)
    F.fq_grouped_gemm_bwd_scale(dh, None, R, layer.seg, layer.shape_gu, layer.w_gu, layer.wfq_gu,
                                layer.q_gu, None, dxq, None, None, layer.ws)
    F.fq_moe_unpermute_reduce(dxq, layer.row_of[:T], x, T, layer.topk, layer.H, layer.aq1, dx2,
                              None, None)
    assert same(bits(dx2, g2, d2), got)
    if learn:
        assert same(bits(dsa), bits(layer.ds_a2))
    # and again, with the input out of its checkpoint
    layer.forward(x, ids, p)
    dx, *_ = layer.backward(None, p, dout)
    xc, xs = O.ckpt_save(host_bits(x), *ckpt)
    assert np.array_equal(host_bits(layer.x_back[:T]), O.ckpt_load(xc, xs, ckpt[0]))
    back = layer.x_back[:T].clone()
    a = bits(dx, layer.ds_gu, layer.ds_d)
    layer.forward(x, ids, p)
    dx, *_ = layer.backward(back, p, dout)
    assert same(a, bits(dx, layer.ds_gu, layer.ds_d))


def test_layers_that_share_their_buffers():
    """Two layers in a row, forward then backward, over one set of buffers: the
    bits of two layers with buffers of their own."""
    ck = (O.FMT_INT8, 128)

    def chain(shared):
        l1, x, ids, p, dout = make(O.FMT_FP8, O.FMT_FP8, None, seed=5, ckpt=ck)
        l2, _, ids2, p2, _ = make(O.FMT_FP8, O.FMT_FP8, None, seed=6, ckpt=ck,
                                  **({"scratch_of": l1} if shared else {}))
        out = []
        for step in range(3):
            for m in (l1, l2):
                m.quantize_weights()
            y = l1.forward(x, ids, p)
            z = l2.forward(y, ids2, p2)
            out += bits(z)
            d2, g2, s2 = l2.backward(None, p2, dout)
            d1, g1, s1 = l1.backward(None, p, d2)
            out += bits(d1, g2, s2, g1, s1)
        return out

    assert same(chain(False), chain(True))


def test_sharing_and_checkpoint_refusals():
    l1, *_ = make(O.FMT_FP8, O.FMT_FP8, None, ckpt=(O.FMT_INT8, 64))
    with pytest.raises(ValueError):
        make(O.FMT_FP8, O.FMT_FP8, None, scratch_of=l1)
    with pytest.raises(ValueError):
        make(O.FMT_FP8, O.FMT_FP8, None, T=71, ckpt=(O.FMT_INT8, 64), scratch_of=l1)
    for ck in ((O.FMT_NVFP4, 16), (O.FMT_INT8, 48), (O.FMT_INT8, 0), (O.FMT_FP8, 512)):
        with pytest.raises(ValueError):
            make(O.FMT_FP8, O.FMT_FP8, None, ckpt=ck)
    plain, x, ids, p, dout = make(O.FMT_FP8, O.FMT_FP8, None)
    with pytest.raises(ValueError):
        plain.backward(None, p, dout)
    with pytest.raises(ValueError):
        plain.forward_tokens(x[:2], ids[:2], p[:2])


@pytest.mark.parametrize("name,wfmt,afmt,group", FORMATS)
def test_export_and_decode(name, wfmt, afmt, group):
    """forward_tokens over the layer's own export, at growing batches, against
    float64 from the layer's quantizer parameters."""
    layer, x, ids, p, _ = make(wfmt, afmt, group)
    gu, d = layer.export()
    vals = []
    for st, w, q in ((gu, layer.w_gu, layer.q_gu), (d, layer.w_d, layer.q_d)):
        host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        vals.append(O.stored_values(host_bits(w), q.fmt, q.group, host(q.scale),
                                    host(q.zero_point), host(q.global_scale)))
    s1, s2 = (float(a.scale) for a in (layer.aq1, layer.aq2))
    for T in (1, 7, 70):
        out = layer.forward_tokens(x[:T], ids[:T], p[:T])
        ref, tol = O.moe_tokens(host_bits(x[:T]), ids[:T].cpu().numpy(), p[:T].cpu().numpy(), 0,
                                *vals, afmt, np.float32(s1), np.float32(s2))
        err = np.abs(bf16_vals(host_bits(out)) - ref)
        assert np.all(err <= tol + 2.0 ** -8 * (np.abs(ref) + tol)), (name, T)
    for bad in ((x[:4], ids[:3], p[:4]), (x[:4], ids[:4], p[:4].half()),
                (x[:4], ids[:4].long(), p[:4]), (x[:4, :128], ids[:4], p[:4]),
                (x[:4].float(), ids[:4], p[:4])):
        with pytest.raises(ValueError):
            layer.forward_tokens(*bad)
    with pytest.raises(F.FQError):
        layer.forward_tokens(x.repeat(2, 1), ids.repeat(2, 1), p.repeat(2, 1))


def test_train_then_decode_in_graphs():
    """A checkpointed training step and a decoding step, each captured once and
    replayed in turn with eager work between: the eager bits."""
    layer, x, ids, p, dout = make(O.FMT_NVFP4, O.FMT_NVFP4, 16, ckpt=(O.FMT_INT8, 64))
    layer.export()

    def train():
        layer.quantize_weights()
        layer.forward(x, ids, p)
        layer.backward(None, p, dout)

    def decode():
        return layer.forward_tokens(x[:5], ids[:5], p[:5])

    train()
    want_t = bits(layer.out, layer.dx, layer.ds_gu, layer.ds_d)
    want_d = bits(decode())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
        decode()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gt, gd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gt):
        train()
    with torch.cuda.graph(gd):
        out = decode()
    for _ in range(3):
        for t in (layer.out, layer.dx, layer.ds_gu, layer.ds_d, out):
            t.zero_()
        gd.replay()
        gt.replay()
        assert same(bits(layer.out, layer.dx, layer.ds_gu, layer.ds_d), want_t)
        assert same(bits(out), want_d)
        decode()
        train()
        layer.forward_tokens(x, ids, p)      # another size, and the export again
        layer.export()
