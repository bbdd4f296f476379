"""Forms of the checkpointed layer and of its decoding that test_gpu_layer_ckpt
does not run."""
import pytest

import oracle as O
from test_gpu_layer_ckpt import bits, make, same

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
