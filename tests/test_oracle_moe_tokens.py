"""Pins of the few-token MoE layer's oracle and the library's refusals of bad
calls (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import oracle as O
from test_abi_host import _no_gpu_visible, pkg  # noqa: F401  (fixture)
from tokens_case import make, reference

host_only = pytest.mark.skipif(not _no_gpu_visible(), reason="placeholder pointers")


@pytest.mark.parametrize("fmt,group", [(O.FMT_INT8, 48), (O.FMT_INT8, O.GROUP_TENSOR),
                                       (O.FMT_FP8, 16), (O.FMT_INT4, 32), (O.FMT_NVFP4, 16),
                                       (O.FMT_NONE, 0)])
def test_stored_values_are_the_fake_quant_values(fmt, group):
    """Within bf16's half step of the decode of an export, and equal to it where
    the definition rounds."""
    c = make(1, 1, 2, 96, 96, 1, fmt, group, O.FMT_NONE)
    for f, g, bits, q in (c["gu"], c["d"]):
        v = O.stored_values(bits, f, g, *q)
        ref = O.bf16_to_f32(O.fq_weight_stack(bits, f, g, *q).bits).astype(np.float64)
        assert np.all(np.abs(v - ref) <= 2.0 ** -8 * np.abs(v) * 1.001)
        if f in (O.FMT_INT8, O.FMT_FP8, O.FMT_INT4) and 0 < g < v.shape[2]:
            assert np.array_equal(v, ref)


@pytest.mark.parametrize("fmt,group,afmt", [(O.FMT_NVFP4, 16, O.FMT_NVFP4),
                                            (O.FMT_FP8, None, O.FMT_FP8),
                                            (O.FMT_INT4, None, O.FMT_NONE),
                                            (O.FMT_INT8, None, O.FMT_INT8)])
def test_against_the_layer_oracle(fmt, group, afmt):
    """The layer's own oracle (bf16 H, A and O, bf16 weights) agrees within the
    roundings it makes: half a bf16 step of h, a and o each, of every weight
    (2^-8 of a sum of magnitudes, entered through rel_h by its ratio here)."""
    c = make(2, 5, 4, 64, 32, 2, fmt, group, afmt)
    (f, g, wg, qg), (_, gd, wd, qd) = c["gu"], c["d"]
    out, tol = reference(c, rel_h=2.0 ** -5)
    x, ids = c["x"], c["ids"]
    ref = np.zeros((c["T"], c["H"]))
    for t in range(c["T"]):
        for j, e in enumerate(ids[t]):
            xq = O.bf16_to_f32(O.fq_act(x[t:t + 1], afmt, c["s1"]).bits).astype(np.float64)
            wv = O.bf16_to_f32(O.fq_weight_stack(wg, f, g, *qg).bits[e]).astype(np.float64)
            h = O.f64_to_bf16(xq @ wv.T)
            aq = O.swiglu_actfq(h, afmt, c["s2"])[1]
            dv = O.bf16_to_f32(O.fq_weight_stack(wd, f, gd, *qd).bits[e]).astype(np.float64)
            ref[t] += float(c["probs"][t, j]) * (
                dv @ O.bf16_to_f32(aq.bits).astype(np.float64)[0])
    assert np.all(np.abs(out - ref) <= tol)
    assert np.all(tol < 2.0 * np.abs(ref).max())


def test_tokens_without_local_experts_and_repeats():
    c = make(3, 4, 2, 32, 16, 3, O.FMT_INT8, None, O.FMT_NONE, E_all=9, begin=4)
    c["ids"][:] = [[0, 1, 2], [4, 4, 5], [-1, 99, 5], [5, 4, 8]]
    out, _ = reference(c)
    assert np.all(out[0] == 0)
    one = dict(c, ids=c["ids"].copy(), probs=c["probs"].copy())
    one["ids"][1] = [4, 0, 5]
    one["probs"][1, 0] = np.float32(c["probs"][1, 0] + c["probs"][1, 1])
    assert np.allclose(reference(one)[0][1], out[1], rtol=1e-6)


@host_only
def test_refusals(pkg):  # noqa: F811
    lib, P = pkg.lib(), 0x1000
    ref = ctypes.byref

    def w(fmt=pkg.FMT_NVFP4, group=16, codes=P, scale=P, sb=P, zp=P, g=P):
        return pkg.fq_stored_w(fmt, group, codes, scale, sb, zp, g)

    def call(x=P, T=4, H=256, F=128, ids=P, probs=P, topk=2, begin=0, E=8, gu=None, d=None, a1=None,
             a2=None, out=P, ws=P, wsb=1 << 40):
        return lib.fq_moe_tokens(x, T, H, F, ids, probs, topk, begin, E, ref(gu or w()),
                                 ref(d or w()), a1, a2, out, ws, wsb, None)

    noscale = ref(pkg.fq_act_q(pkg.FMT_FP8_E4M3, None))
    arg = pkg.FQ_ERR_INVALID_ARGUMENT
    for bad in (dict(x=None), dict(ids=None), dict(probs=None), dict(out=None), dict(T=-1),
                dict(H=0), dict(F=-16), dict(topk=0), dict(E=0), dict(begin=-1),
                dict(begin=2 ** 31 - 4), dict(x=P + 8), dict(out=P + 2), dict(a1=noscale),
                dict(a2=noscale), dict(gu=w(fmt=9)), dict(gu=w(codes=None)), dict(d=w(codes=P + 8)),
                dict(gu=w(group=32)), dict(gu=w(sb=None)), dict(d=w(g=None)), dict(d=w(sb=P + 8)),
                dict(gu=w(pkg.FMT_INT8, 256, scale=None)), dict(gu=w(pkg.FMT_INT8, 256, scale=P + 4)),
                dict(gu=w(pkg.FMT_INT4, 128, zp=P + 1)), dict(gu=w(pkg.FMT_INT4, 128, zp=None)),
                dict(gu=w(pkg.FMT_INT4, -1)), dict(gu=w(pkg.FMT_INT8, 96)),
                dict(gu=w(pkg.FMT_FP8_E4M3, 24)), dict(gu=w(pkg.FMT_INT8, 0)), dict(ws=P + 8)):
        assert call(**bad) == arg, bad
        assert lib.fq_last_error()
    for bad in (dict(T=129), dict(topk=65), dict(E=1025), dict(H=264), dict(F=136), dict(H=16400),
                dict(F=16400), dict(gu=w(pkg.FMT_INT4, 16)), dict(d=w(pkg.FMT_INT4, 16))):
        assert call(**bad) == pkg.FQ_ERR_UNSUPPORTED, bad
    # scales that do not fit into LDS, whatever the rest
    for H, gu in ((16384, w(pkg.FMT_INT8, 16)), (16368, w(pkg.FMT_FP8_E4M3, 16))):
        assert call(H=H, F=64, gu=gu, d=w()) == pkg.FQ_ERR_UNSUPPORTED
        assert b"LDS" in lib.fq_last_error()
    assert lib.fq_moe_tokens(P, 4, 256, 128, P, P, 2, 0, 8, None, ref(w()), None, None, P, P,
                             1 << 40, None) == arg
    need = pkg.fq_workspace_bytes(pkg.FQ_OP_MOE_TOKENS, (8, 256, 128), 8, 2)
    assert need > 0
    assert call(wsb=need - 1) == pkg.FQ_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=None) == pkg.FQ_ERR_WORKSPACE_TOO_SMALL
    # nothing to do: no launch, no workspace
    assert call(T=0, x=None, ids=None, probs=None, out=None, ws=None, wsb=0) == pkg.FQ_OK
    for shape, R, k in (((0, 256, 128), 8, 2), ((8, 256, 128), 8, 0), ((8, 256, 128), 7, 2),
                        ((8, 256, 128), -2, 2)):
        assert pkg.fq_workspace_bytes(pkg.FQ_OP_MOE_TOKENS, shape, R, k) == 0


@host_only
def test_workspace_holds_every_buffer(pkg):  # noqa: F811
    """The A rows and the rows' tokens and weights, at the ends of the range."""
    for T in (1, 2, 7, 64, 128):
        for topk in (1, 8, 64):
            for E, H, Fc in ((1, 16, 16), (128, 2048, 768), (1024, 16384, 16384)):
                P = T * topk
                slots = min(P, E)
                got = pkg.fq_workspace_bytes(pkg.FQ_OP_MOE_TOKENS, (E, H, Fc), P, topk)
                assert got >= P * Fc * 2 + slots * 16 + P * 8
