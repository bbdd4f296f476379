"""GPU parity of the few-token MoE layer over stored weights through the C ABI,
against float64 with a bound that counts fp32 sums, quantizer borders and the
rounding of the output (half a bf16 step)."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import bf16_vals, dev_bf16, dev_f32, dev_i32, host_bits
from tokens_case import make, reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None


def stored(fmt, group, bits, q):
    """The exported stack on the device, its codes packed by the oracle."""
    if fmt == O.FMT_NONE:
        return F.StoredW(fmt, 0, dev_bf16(bits))
    s, zp, g = q
    code = O.fq_weight_stack(bits, fmt, group, s, zp, g).code
    st = F.StoredW(fmt, group, torch.from_numpy(np.ascontiguousarray(
        O.pack_codes(code, fmt))).cuda())
    _, sb, zb = O.export_scales(fmt, s, zp)
    if fmt == O.FMT_NVFP4:
        st.scale_bytes, st.global_scale = torch.from_numpy(sb.reshape(-1)).cuda(), dev_f32(g)
    else:
        st.scale = dev_f32(s)
        if fmt == O.FMT_INT4:
            st.zero_point_bytes = torch.from_numpy(zb.reshape(-1)).cuda()
    return st


class Call:
    def __init__(self, c):
        self.c = c
        self.gu, self.d = stored(*c["gu"]), stored(*c["d"])
        self.x, self.ids, self.p = dev_bf16(c["x"]), dev_i32(c["ids"]), dev_f32(c["probs"])
        self.a1 = F.ActQ(c["afmt"], dev_f32([c["s1"]]))
        self.a2 = F.ActQ(c["afmt"], dev_f32([c["s2"]]))
        n = F.fq_workspace_bytes(F.FQ_OP_MOE_TOKENS, (c["E"], c["H"], c["F"]), c["T"] * c["topk"],
                                 c["topk"])
        # exactly the documented size, the bytes behind it watched
        self.buf = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        self.ws = self.buf[:n]
        self.out = torch.full((c["T"] + 1, c["H"]), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self):
        c = self.c
        F.fq_moe_tokens(self.x, c["T"], c["H"], c["F"], self.ids, self.p, c["topk"], c["begin"],
                        c["E"], self.gu, self.d, self.a1, self.a2, self.out[:c["T"]], self.ws)

    def check(self, against=None):
        ref, tol = against or reference(self.c)
        torch.cuda.synchronize()
        got = bf16_vals(host_bits(self.out))
        T = self.c["T"]
        err = np.abs(got[:T] - ref)
        lim = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133
        assert np.all(err <= lim), f"worst {np.max(err / np.maximum(lim, 1e-30)):.3g} of the bound"
        assert np.all(got[T:] == 7.0) and bool((self.buf[self.ws.numel():] == 0x5A).all())
        return float((err / np.abs(ref).max()).max()) if ref.any() else 0.0


def run_case(**kw):
    call = Call(make(**kw))
    print(f"[tokens] {kw}", flush=True)
    call.run()
    rel = call.check()
    print(f"[tokens] max|err|/max|ref| {rel:.3g}", flush=True)
    return call


FORMATS = [(O.FMT_NVFP4, 16, O.FMT_NVFP4), (O.FMT_NVFP4, 16, O.FMT_NONE),
           (O.FMT_FP8, None, O.FMT_FP8), (O.FMT_FP8, O.GROUP_TENSOR, O.FMT_FP8),
           (O.FMT_FP8, 64, O.FMT_NONE), (O.FMT_FP8, 16, O.FMT_FP8),
           (O.FMT_INT4, 128, O.FMT_NONE), (O.FMT_INT4, 32, O.FMT_FP8),
           (O.FMT_INT4, None, O.FMT_NONE), (O.FMT_INT8, None, O.FMT_INT8),
           (O.FMT_INT8, 128, O.FMT_INT8), (O.FMT_INT8, 32, O.FMT_NONE),
           (O.FMT_INT8, O.GROUP_TENSOR, O.FMT_INT8), (O.FMT_NONE, 0, O.FMT_NONE)]


@pytest.mark.parametrize("fmt,group,afmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 33])
def test_formats(fmt, group, afmt, T):
    """Fewer pairs than experts (T = 1), about as many, and several per expert."""
    run_case(seed=10 + T, T=T, E=12, H=256, F=128, topk=3, fmt=fmt, group=group, afmt=afmt)


@pytest.mark.parametrize("fmt,group,afmt", [f for f in FORMATS if f[1] not in (64, 128, 32)])
@pytest.mark.parametrize("H,Fc", [(16, 16), (272, 208), (1040, 48), (48, 368)])
def test_odd_sizes(fmt, group, afmt, H, Fc):
    """Rows that end inside a load (K % 32 = 16), a chunk or a wave's share."""
    run_case(seed=30, T=4, E=5, H=H, F=Fc, topk=2, fmt=fmt, group=group, afmt=afmt)


@pytest.mark.parametrize("fmt,group,H,Fc", [(O.FMT_INT4, 96, 288, 192), (O.FMT_INT8, 48, 144, 96),
                                            (O.FMT_INT4, 256, 512, 256), (O.FMT_FP8, 192, 384, 192)])
def test_odd_groups(fmt, group, H, Fc):
    run_case(seed=31, T=3, E=4, H=H, F=Fc, topk=2, fmt=fmt, group=group, afmt=O.FMT_NONE)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 48, 127, 128])
def test_token_counts(T):
    run_case(seed=40 + T, T=T, E=16, H=512, F=64, topk=4, fmt=O.FMT_NVFP4, group=16,
             afmt=O.FMT_NVFP4)


def test_every_token_on_one_expert():
    """128 columns of one expert: several column groups, the others idle."""
    c = make(seed=50, T=128, E=6, H=1024, F=96, topk=1, fmt=O.FMT_INT8, group=None, afmt=O.FMT_INT8)
    c["ids"][:] = 4
    call = Call(c)
    call.run()
    call.check()


@pytest.mark.parametrize("fmt,group,afmt", [(O.FMT_NVFP4, 16, O.FMT_NVFP4),
                                            (O.FMT_INT4, 128, O.FMT_NONE)])
def test_hot_expert_among_others(fmt, group, afmt):
    """Most tokens share one expert (several passes of columns), the rest name
    others: the blocks' shares fall inside experts of different weight."""
    c = make(seed=57, T=100, E=40, H=1024, F=256, topk=3, fmt=fmt, group=group, afmt=afmt)
    c["ids"][:90, 1] = 17
    c["ids"][90:, 2] = 39
    call = Call(c)
    call.run()
    call.check()
    first = call.out.clone()
    call.ws.fill_(0xFF)              # nothing is kept in the workspace
    call.run()
    assert torch.equal(call.out, first)


def test_wide_rows_stage_few_columns():
    """A row so wide that fewer than 16 token rows fit into LDS at a time."""
    run_case(seed=51, T=9, E=2, H=8192, F=32, topk=1, fmt=O.FMT_FP8, group=None, afmt=O.FMT_FP8)
    run_case(seed=52, T=3, E=1, H=16384, F=16, topk=1, fmt=O.FMT_NVFP4, group=16, afmt=O.FMT_NONE)


def test_wide_rows_of_small_groups_and_many_pairs():
    """The largest use of LDS: an expert row's scales and zero points, and the
    pairs of 128 tokens that name 64 experts each."""
    run_case(seed=55, T=2, E=1, H=16384, F=32, topk=1, fmt=O.FMT_INT4, group=32, afmt=O.FMT_NONE)
    run_case(seed=56, T=128, E=70, H=64, F=32, topk=64, fmt=O.FMT_INT8, group=None,
             afmt=O.FMT_INT8)


def test_wide_f():
    run_case(seed=53, T=3, E=2, H=32, F=4096, topk=2, fmt=O.FMT_INT4, group=None, group_d=128,
             afmt=O.FMT_NONE)


def test_mixed_formats():
    run_case(seed=54, T=6, E=4, H=256, F=128, topk=2, fmt=O.FMT_NVFP4, group=16, afmt=O.FMT_NONE,
             fmt_d=O.FMT_INT8, group_d=128)


@pytest.mark.parametrize("T,topk", [(4, 3), (40, 3)])
def test_local_share_repeats_and_foreign_ids(T, topk):
    """One rank's experts: foreign ids, ids that exist nowhere, a token without
    a local expert (its row is 0), a token that names an expert twice."""
    c = make(seed=60, T=T, E=20, H=128, F=64, topk=topk, fmt=O.FMT_FP8, group=None, afmt=O.FMT_FP8,
             E_all=64, begin=30)
    c["ids"][0] = [29, 50, 0]
    c["ids"][1] = [31, 31, 31]
    c["ids"][2] = [-1, 2 ** 31 - 1, 49]
    c["ids"][3] = [35, -2 ** 31, 35]
    call = Call(c)
    call.run()
    call.check()
    assert not call.out[0].any()


def test_no_local_pair_at_all():
    c = make(seed=61, T=7, E=4, H=64, F=32, topk=2, fmt=O.FMT_INT8, group=None, afmt=O.FMT_NONE)
    c["ids"][:] = 99
    call = Call(c)
    call.run()
    assert not call.out[:7].any()


def test_many_experts():
    """1024 experts, more pairs than experts and fewer."""
    for T in (3, 128):
        run_case(seed=62, T=T, E=1024, H=32, F=16, topk=9, fmt=O.FMT_INT8, group=None,
                 afmt=O.FMT_NONE)


def test_non_finite_inputs_stay_in_their_rows():
    c = make(seed=63, T=4, E=3, H=128, F=64, topk=2, fmt=O.FMT_INT8, group=None, afmt=O.FMT_NONE)
    good = Call(c)
    good.run()
    c = dict(c, x=c["x"].copy(), probs=c["probs"].copy())
    c["x"][1, 5], c["x"][2, 7] = 0x7FC0, 0x7F80
    bad = Call(c)
    bad.run()
    nan = torch.isnan(bad.out.float()).cpu().numpy()
    assert nan[1].all()
    assert not nan[[0, 3]].any()
    assert torch.equal(bad.out[[0, 3]], good.out[[0, 3]])


def test_same_bits_again_other_stream_and_replay():
    """Repeated, on another stream, and replayed from a graph with other calls
    over the same workspace in between."""
    call = Call(make(seed=70, T=21, E=24, H=256, F=128, topk=4, fmt=O.FMT_NVFP4, group=16,
                     afmt=O.FMT_NVFP4))
    small = Call(make(seed=71, T=2, E=24, H=256, F=128, topk=4, fmt=O.FMT_NVFP4, group=16,
                      afmt=O.FMT_NVFP4))
    small.ws = call.ws
    call.run()
    want = call.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call.run()
    side.synchronize()
    assert torch.equal(call.out[:21], want[:21])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    small.run()
    torch.cuda.synchronize()
    sw = small.out.clone()
    for _ in range(4):
        call.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out[:21], want[:21])
        small.out.zero_()
        small.run()
        call.ws.fill_(0xFF)
        torch.cuda.synchronize()
        assert torch.equal(small.out[:2], sw[:2])


def test_two_streams_with_workspaces_of_their_own():
    a = Call(make(seed=72, T=16, E=8, H=512, F=256, topk=2, fmt=O.FMT_FP8, group=None,
                  afmt=O.FMT_FP8))
    b = Call(make(seed=73, T=9, E=8, H=512, F=256, topk=2, fmt=O.FMT_INT4, group=128,
                  afmt=O.FMT_NONE))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_default_workload_layer():
    """H 2048, F 768, top 8: eight experts alone, and the same eight scattered
    among 128 (every expert's codes at its own offset)."""
    rng = np.random.default_rng(80)
    for T in (1, 9):
        c = make(seed=81, T=T, E=8, H=2048, F=768, topk=8, fmt=O.FMT_NVFP4, group=16,
                 afmt=O.FMT_NVFP4)
        ref = reference(c)
        small = Call(c)
        small.run()
        small.check(ref)
        place = np.sort(rng.choice(128, 8, replace=False))
        at = torch.from_numpy(place).cuda()
        big = Call(c)
        for st, per in ((big.gu, 2 * 768 * 2048), (big.d, 2048 * 768)):
            for name, n in (("codes", per // 2), ("scale_bytes", per // 16), ("global_scale", 1)):
                src = getattr(st, name).reshape(8, n)
                dst = torch.full((128, n), 0x22, dtype=torch.uint8, device="cuda").to(src.dtype)
                dst[at] = src
                setattr(st, name, dst.reshape(-1))
        big.ids = dev_i32(place[c["ids"]])
        F.fq_moe_tokens(big.x, T, 2048, 768, big.ids, big.p, 8, 0, 128, big.gu, big.d, big.a1,
                        big.a2, big.out[:T], torch.empty(
                            F.fq_workspace_bytes(F.FQ_OP_MOE_TOKENS, (128, 2048, 768), T * 8, 8),
                            dtype=torch.uint8, device="cuda"))
        big.check(ref)


def test_refusals_with_device_tensors():
    call = Call(make(seed=90, T=2, E=2, H=32, F=16, topk=1, fmt=O.FMT_INT8, group=None,
                     afmt=O.FMT_NONE))
    call.ws = call.ws[:-256]
    with pytest.raises(F.FQError) as e:
        call.run()
    assert e.value.status == F.FQ_ERR_WORKSPACE_TOO_SMALL
    call.c = dict(call.c, T=129)
    with pytest.raises(F.FQError) as e:
        call.run()
    assert e.value.status == F.FQ_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        F.fq_moe_tokens(call.x.cpu(), 2, 32, 16, call.ids, call.p, 1, 0, 2, call.gu, call.d,
                        call.a1, call.a2, call.out, call.ws)
