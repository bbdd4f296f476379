"""GPU parity of forms of the few-token MoE layer that test_gpu_moe_tokens does
not launch, by the same bound."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import dev_bf16, dev_f32, dev_i32
from test_gpu_moe_tokens import Call, F, make, run_case
from test_oracle_moe_tokens_a import FORMS, SMALL_GROUPS, difference_case
from tokens_case import reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group", FORMS)
@pytest.mark.parametrize("T", [1, 20])
def test_a_without_an_activation_format_is_not_rounded(fmt, group, T):
    """Outputs that are differences of A below a bf16 step of A."""
    print(f"[tokens] differences fmt={fmt} group={group} T={T}", flush=True)
    call = Call(difference_case(100 + T, T, 3, 256, 256, fmt, group))
    call.run()
    call.check()


@pytest.mark.parametrize("fmt,group", SMALL_GROUPS)
@pytest.mark.parametrize("T", [1, 20])
def test_weights_of_small_groups_are_not_rounded(fmt, group, T):
    """Groups whose scales are no bf16 numbers, in rows that whole and ended chunks make."""
    for H, Fc in ((256, 256), (288 if group == 32 else 208 if group == 16 else 320, 128)):
        print(f"[tokens] weights fmt={fmt} group={group} T={T} H={H}", flush=True)
        call = Call(difference_case(130 + T, T, 3, H, Fc, fmt, group, uneven=True))
        call.run()
        call.check()


def test_a_beyond_the_largest_bf16_number():
    """A between the largest bf16 and the largest fp32 number, and infinite."""
    H, Fc = 32, 16
    c = make(seed=101, T=3, E=1, H=H, F=Fc, topk=1, fmt=O.FMT_NONE, group=0, afmt=O.FMT_NONE)
    gu = np.zeros((1, 2 * Fc, H), np.float32)
    gu[0, :, 0] = 1.0                       # h = x[0] for the gate rows,
    gu[0, Fc:, 0], gu[0, Fc:, 1] = 0.0, 1.0  # x[1] for the up rows
    d = np.full((1, H, Fc), 2.0 ** -10, np.float32)
    x = np.zeros((3, H), np.float32)
    x[:, 0] = 256.0                         # silu(256) = 256
    x[0, 0], x[0, 1] = 362.0, 181 * 2.0 ** 112  # A = 1.9996 2^127: infinite as one bf16 number
    x[1, 1] = 2.0 ** 120                    # A = 2^128
    x[2, 1] = -1.0
    c["gu"] = (O.FMT_NONE, 0, O.f32_to_bf16(gu), (None,) * 3)
    c["d"] = (O.FMT_NONE, 0, O.f32_to_bf16(d), (None,) * 3)
    c["x"] = O.f32_to_bf16(x)
    c["probs"][:] = 1.0
    a0 = 362.0 * 181 * 2.0 ** 112
    assert float.fromhex("0x1.FFp127") < a0 < 2.0 ** 128
    call = Call(c)
    call.run()
    got = call.out[:3].double().cpu().numpy()
    assert np.all(np.abs(got[0] - Fc * 2.0 ** -10 * a0) <= 2.0 ** -8 * Fc * 2.0 ** -10 * a0)
    assert np.all(np.isposinf(got[1]))
    assert np.all(np.abs(got[2] + Fc * 2.0 ** -10 * 256.0) <= 2.0 ** -8 * Fc * 0.25)


@pytest.mark.parametrize("fmt,group,afmt,H", [(O.FMT_INT8, 16, O.FMT_INT8, 8400),
                                              (O.FMT_FP8, 16, O.FMT_NONE, 15136),
                                              (O.FMT_FP8, 16, O.FMT_FP8, 15104),
                                              (O.FMT_INT4, 32, O.FMT_NONE, 16352)])
def test_wide_rows_of_small_groups(fmt, group, afmt, H):
    """Scale rows that fit into LDS for one channel group only, rows that end
    inside a chunk and whole ones, up to the widest accepted."""
    run_case(seed=110, T=3, E=2, H=H, F=32, topk=1, fmt=fmt, group=group, afmt=afmt)


def channel_groups(c):
    """The channel groups of a gate_up item (whole rows), by the launch's rule."""
    fmt, group = c["gu"][0], c["gu"][1]
    chunk = {O.FMT_NONE: 32, O.FMT_INT8: 64, O.FMT_FP8: 64}.get(c["d"][0], 128)
    groups = -(-c["F"] // chunk) * chunk // 16
    slots = min(c["T"] * c["topk"], c["E"])
    mt = 4
    while mt > 1 and slots * -(-groups // mt) < 1024:
        mt //= 2
    ng = c["H"] // group if group > 0 else 0
    up = lambda n: (n + 7) // 8 * 8 + 8  # noqa: E731
    row = up(c["H"] // 16) if fmt == O.FMT_NVFP4 else up(4 * ng) if ng > 1 else 0
    row += up(ng) if fmt == O.FMT_INT4 else 0
    while mt > 1 and 2 * mt * 16 * row > 20480:
        mt //= 2
    return mt


def tiled(c, times, ids):
    """The call over `times` copies of the experts, expert e at e, e + E, ...:
    a stack of many experts whose float64 form is that of a few."""
    E = c["E"]
    call = Call(dict(c, E=E * times, ids=ids))
    for st in (call.gu, call.d):
        for name in ("codes", "scale", "scale_bytes", "zero_point_bytes", "global_scale"):
            t = getattr(st, name)
            if t is not None:
                setattr(st, name, t.reshape(E, -1).repeat(times, 1).reshape(-1))
    return call, reference(dict(c, ids=ids % E))


WIDE_ITEMS = [(O.FMT_NVFP4, 16, O.FMT_NVFP4, 1152), (O.FMT_NVFP4, 16, O.FMT_NONE, 1152),
              (O.FMT_FP8, None, O.FMT_FP8, 1152), (O.FMT_FP8, O.GROUP_TENSOR, O.FMT_FP8, 1152),
              (O.FMT_FP8, 64, O.FMT_NONE, 1152), (O.FMT_FP8, 16, O.FMT_FP8, 576),
              (O.FMT_INT4, 128, O.FMT_NONE, 1152), (O.FMT_INT4, 32, O.FMT_FP8, 768),
              (O.FMT_INT4, None, O.FMT_NONE, 1152), (O.FMT_INT8, None, O.FMT_INT8, 1152),
              (O.FMT_INT8, 192, O.FMT_INT8, 1152), (O.FMT_INT8, 32, O.FMT_NONE, 1152),
              (O.FMT_INT8, O.GROUP_TENSOR, O.FMT_INT8, 1152), (O.FMT_NONE, 0, O.FMT_NONE, 1152)]


@pytest.mark.parametrize("fmt,group,afmt,H", WIDE_ITEMS)
@pytest.mark.parametrize("mt", [4, 2])
def test_items_of_several_channel_groups(fmt, group, afmt, H, mt):
    """Enough experts for items of 64 and of 32 channels, F = 17 x 16 that ends
    inside an item, contractions of several rounds of the waves, and an expert
    of more rows than one pass stages."""
    topk = 2 * mt
    c = make(seed=120 + mt, T=32, E=8, H=H, F=272, topk=topk, fmt=fmt, group=group,
             group_d=272 if group and group > 16 else None, afmt=afmt)
    ids = np.stack([np.random.default_rng(t).permutation(256)[:topk] for t in range(32)])
    ids[:20, 0] = 17
    call, ref = tiled(c, 32, ids.astype(np.int32))
    assert channel_groups(call.c) == mt
    print(f"[tokens] {mt} channel groups fmt={fmt} group={group} afmt={afmt} H={H}", flush=True)
    call.run()
    call.check(ref)


@pytest.mark.parametrize("fmt,afmt", [(O.FMT_FP8, O.FMT_FP8), (O.FMT_INT8, O.FMT_NONE)])
def test_wide_rows_of_small_groups_two_channel_groups(fmt, afmt):
    """Rows that end inside a chunk, 64 of them with their scales in LDS."""
    run_case(seed=111, T=9, E=3, H=4112, F=48, topk=2, fmt=fmt, group=16, afmt=afmt)


ACTS = {O.FMT_NONE: 1.0, O.FMT_FP8: 448.0, O.FMT_INT8: 127.0, O.FMT_NVFP4: 2688.0}
CROSSED = [(O.FMT_NVFP4, 16, O.FMT_NVFP4, O.FMT_NONE), (O.FMT_NVFP4, 16, O.FMT_NONE, O.FMT_NVFP4),
           (O.FMT_NVFP4, 16, O.FMT_FP8, O.FMT_INT8), (O.FMT_NVFP4, 16, O.FMT_INT8, O.FMT_FP8),
           (O.FMT_INT8, None, O.FMT_NVFP4, O.FMT_NVFP4), (O.FMT_INT8, 32, O.FMT_FP8, O.FMT_NONE),
           (O.FMT_FP8, 64, O.FMT_NONE, O.FMT_INT8), (O.FMT_FP8, O.GROUP_TENSOR, O.FMT_INT8, O.FMT_NVFP4),
           (O.FMT_INT4, 64, O.FMT_NVFP4, O.FMT_INT8), (O.FMT_INT4, 128, O.FMT_INT8, O.FMT_NVFP4),
           (O.FMT_NONE, 0, O.FMT_FP8, O.FMT_NVFP4), (O.FMT_NONE, 0, O.FMT_NVFP4, O.FMT_FP8)]


@pytest.mark.parametrize("fmt,group,a1,a2", CROSSED)
def test_activation_formats_of_their_own(fmt, group, a1, a2):
    """Weights under another format's activations, x and A in different ones."""
    print(f"[tokens] fmt={fmt} group={group} a1={a1} a2={a2}", flush=True)
    c = make(seed=140, T=11, E=6, H=256, F=128, topk=3, fmt=fmt, group=group, afmt=O.FMT_NONE)
    c["s1"] = np.float32(c["s1"] / ACTS[a1])
    c["s2"] = np.float32(c["s2"] / ACTS[a2])
    call = Call(c)
    call.a1, call.a2 = F.ActQ(a1, dev_f32([c["s1"]])), F.ActQ(a2, dev_f32([c["s2"]]))
    call.run()
    vals = [O.stored_values(bits, f, g, *q) for f, g, bits, q in (c["gu"], c["d"])]
    call.check(O.moe_tokens(c["x"], c["ids"], c["probs"], 0, *vals, a1, c["s1"], c["s2"], afmt2=a2))


@pytest.mark.parametrize("fmt,group,afmt", [(O.FMT_NVFP4, 16, O.FMT_NVFP4),
                                            (O.FMT_INT4, 32, O.FMT_NONE)])
def test_replays_with_new_tokens(fmt, group, afmt):
    """One captured call, its tokens, routing and weights overwritten between the
    replays (other experts, a hot one, none local at all), eager calls of another
    size over the same workspace in between."""
    c = make(seed=150, T=23, E=24, H=256, F=128, topk=4, fmt=fmt, group=group, afmt=afmt)
    call, eager = Call(c), Call(c)
    small = Call(dict(c, T=2, x=c["x"][:2], ids=c["ids"][:2], probs=c["probs"][:2]))
    small.ws = call.ws
    call.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    rng = np.random.default_rng(151)
    for step in range(5):
        ids = np.stack([rng.permutation(24)[:4] for _ in range(23)]).astype(np.int32)
        if step == 1:
            ids[:, 2] = 5
        if step == 3:
            ids[:] = 24
        new = (dev_bf16(O.f32_to_bf16(rng.standard_normal((23, 256)).astype(np.float32))),
               dev_i32(ids), dev_f32(rng.uniform(0.1, 1.0, (23, 4)).astype(np.float32)))
        for k in (call, eager):
            for to, v in zip((k.x, k.ids, k.p), new):
                to.copy_(v)
        call.out.fill_(7.0)
        g.replay()
        eager.run()
        torch.cuda.synchronize()
        assert torch.equal(call.out.view(torch.int16), eager.out.view(torch.int16)), step
        assert bool(eager.out[:23].any()) == (step != 3)
        small.run()
        call.ws.fill_(0xFF)
        torch.cuda.synchronize()
