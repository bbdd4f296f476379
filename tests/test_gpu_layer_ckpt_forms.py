"""Forms of the checkpointed layer and of its decoding that test_gpu_layer_ckpt
does not run."""
import numpy as np
import pytest

import oracle as O
from helpers import bf16_vals, host_bits
from test_gpu_layer_ckpt import F, bits, make, same

pytestmark = pytest.mark.gpu


def test_an_input_that_was_overwritten_is_refused():
    """The second layer's input is the first one's out, which the second forward
    writes over where the layers share their buffers."""
    ck = (O.FMT_INT8, 64)
    l1, x, ids, p, dout = make(O.FMT_FP8, O.FMT_FP8, None, seed=5, ckpt=ck)
    l2, _, ids2, p2, _ = make(O.FMT_FP8, O.FMT_FP8, None, seed=6, ckpt=ck, scratch_of=l1)
    for m in (l1, l2):
        m.quantize_weights()
    y = l1.forward(x, ids, p)
    keep = y.clone()
    l2.forward(y, ids2, p2)
    for stale in (y, l1.out, l2.out[3:], y.view(-1, 2 * l1.H), l1.dx, l1.xq_tok):
        with pytest.raises(ValueError, match="overwritten"):
            l2.backward(stale, p2, dout)
    want = bits(*l2.backward(keep, p2, dout))
    # the same with buffers of its own, whose input then is another's
    l3, *_ = make(O.FMT_FP8, O.FMT_FP8, None, seed=6, ckpt=ck)
    l3.quantize_weights()
    l3.forward(keep, ids2, p2)
    assert same(bits(*l3.backward(keep, p2, dout)), want)
    with pytest.raises(ValueError, match="overwritten"):
        l3.backward(l3.out, p2, dout)
    # refused before anything ran
    assert same(bits(l3.dx, l3.ds_gu, l3.ds_d), want)


@pytest.mark.parametrize("afmt", [O.FMT_NONE, O.FMT_INT8])
@pytest.mark.parametrize("overlap", [False, True])
@pytest.mark.parametrize("restore", [False, True])
def test_shared_buffers_in_other_forms(afmt, overlap, restore):
    """Without an activation format (the input itself is the gate_up operand, and
    the second layer's lies in the buffer that its forward writes), without the
    second stream, and with the first layer's input given or out of its
    checkpoint: the bits of layers with buffers of their own."""
    wfmt, group = (O.FMT_INT4, 128) if afmt == O.FMT_NONE else (O.FMT_INT8, None)
    ck = (O.FMT_FP8, 64)

    def chain(shared):
        l1, x, ids, p, dout = make(wfmt, afmt, group, seed=15, ckpt=ck)
        l2, _, ids2, p2, _ = make(wfmt, afmt, group, seed=16, ckpt=ck,
                                  **({"scratch_of": l1} if shared else {}))
        out = []
        for m in (l1, l2):
            m.overlap_wgrad = overlap
            m.quantize_weights()
        for step in range(2):
            z = l2.forward(l1.forward(x, ids, p), ids2, p2)
            out += bits(z)
            d2, g2, s2 = l2.backward(None, p2, dout)
            d1, g1, s1 = l1.backward(None if restore else x, p, d2)
            out += bits(d1, g2, s2, g1, s1)
        return out

    assert same(chain(False), chain(True))


@pytest.mark.parametrize("fmt", [O.FMT_INT8, O.FMT_FP8])
def test_export_and_decode_with_one_scale_per_matrix(fmt):
    layer, x, ids, p, _ = make(fmt, fmt, F.FQ_GROUP_TENSOR)
    vals = []
    for st, w, q in zip(layer.export(), (layer.w_gu, layer.w_d), (layer.q_gu, layer.q_d)):
        assert st.group == F.FQ_GROUP_TENSOR and st.scale.numel() == layer.E
        vals.append(O.stored_values(host_bits(w), q.fmt, q.group, q.scale.cpu().numpy()))
    s1, s2 = (np.float32(float(a.scale)) for a in (layer.aq1, layer.aq2))
    for T in (1, 70):
        out = layer.forward_tokens(x[:T], ids[:T], p[:T])
        ref, tol = O.moe_tokens(host_bits(x[:T]), ids[:T].cpu().numpy(), p[:T].cpu().numpy(), 0,
                                *vals, fmt, s1, s2)
        err = np.abs(bf16_vals(host_bits(out)) - ref)
        assert np.all(err <= tol + 2.0 ** -8 * (np.abs(ref) + tol)), T
