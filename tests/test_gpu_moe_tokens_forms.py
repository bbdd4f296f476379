"""GPU parity of forms of the few-token MoE layer that test_gpu_moe_tokens does
not launch, by the same bound."""
import numpy as np
import pytest

import oracle as O
from test_gpu_moe_tokens import Call, make, run_case
from test_oracle_moe_tokens_a import FORMS, difference_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group", FORMS)
@pytest.mark.parametrize("T", [1, 20])
def test_a_without_an_activation_format_is_not_rounded(fmt, group, T):
    """Outputs that are differences of A below a bf16 step of A."""
    print(f"[tokens] differences fmt={fmt} group={group} T={T}", flush=True)
    call = Call(difference_case(100 + T, T, 3, 256, 256, fmt, group))
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
