"""Every form of the int8 and gated products against float64, each case with the form that it
is meant to reach: whole and cut last stages, contractions of one stage, more tiles than blocks."""
import pytest
import torch

import oracle as O
import test_gpu_products as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

ROWS, MID64, MID128, TILE256 = range(4)
BLOCKS64 = 512    # blocks of the 64 x 64 form, and of the 128 x 128 form beyond one tile a CU


def form(kind, E, columns, row_bytes, R):
    return F.lib().fq_internal_product_form(kind, E, columns, row_bytes, R)


def tiles(E, R, columns, side):
    """Tiles of a call whose rows are spread evenly."""
    return E * -(-(R // E) // side) * -(-columns // side)


# (form, E, T, topk, 2F or N, contraction, spare rows, skewed routing); the contraction in bytes
# is the number for int8 and twice it for bf16
CASES = [
    (MID64, 4, 700, 2, 544, 256, 0, False),         # whole stages
    (MID64, 4, 700, 2, 544, 272, 5, True),          # a last stage of 16 (32) bytes
    (MID64, 2, 512, 1, 4096, 128, 0, False),
    (MID64, 3, 260, 3, 608, 2064, 7, False),        # many stages
    (MID64, 64, 256, 4, 1024, 144, 0, False),       # more tiles than blocks
    (MID64, 128, 700, 3, 1056, 64, 9, True),
    (MID64, 130, 520, 4, 512, 32, 0, False),        # one stage, cut
    (MID128, 32, 3200, 3, 768, 144, 0, False),      # more tiles than blocks
    (MID128, 32, 3200, 3, 768, 128, 60, True),
    (MID128, 16, 700, 3, 1056, 64, 0, False),       # one stage (int8: cut)
    (MID128, 8, 1000, 3, 1024, 640, 0, False),
    (TILE256, 64, 1300, 4, 2048, 128, 0, False),    # one stage for int8, two for bf16; several tiles a block
    (TILE256, 64, 1300, 4, 2080, 64, 60, True),     # half a stage, and one
    (TILE256, 64, 1300, 4, 2080, 384, 0, False),    # three and six stages
    (TILE256, 16, 2500, 2, 2080, 256, 9, True),
    (TILE256, 8, 4100, 1, 3104, 1024, 0, False),
]
SECOND = [c for c in CASES if c[0] in (MID64, MID128) and
          tiles(c[1], c[2] * c[3], c[4], 64 if c[0] == MID64 else 128) > BLOCKS64]
IDS = ["-".join(str(v) for v in c[:6]) for c in CASES]


def test_some_cases_have_more_tiles_than_blocks():
    assert {c[0] for c in SECOND} == {MID64, MID128}


@pytest.mark.parametrize("want,E,T,topk,N,K,spare,skew", CASES, ids=IDS)
@pytest.mark.parametrize("routed", [False, True])
def test_int8(want, E, T, topk, N, K, spare, skew, routed):
    assert form(0, E, N, K, T * topk) == want
    base.test_int8_product_bitexact(E, T, topk, N, K, spare, skew, routed, not routed)


# the gated kinds have half the columns of a tile: N is 2F, and the rule counts F in halves
@pytest.mark.parametrize("want,E,T,topk,N,K,spare,skew", CASES, ids=IDS)
def test_gated_int8(want, E, T, topk, N, K, spare, skew):
    assert form(1, E, N // 2, K, T * topk) == want
    base.test_int8_gated_product(E, T, topk, N, K, spare, skew)


@pytest.mark.parametrize("afmt,as_", base.ACTS)
@pytest.mark.parametrize("want,E,T,topk,N,H,spare,skew", CASES, ids=IDS)
def test_gated(want, E, T, topk, N, H, spare, skew, afmt, as_):
    assert form(1, E, N // 2, 2 * H, T * topk) == want
    base.test_gated_forward(E, T, topk, H, N // 2, spare, skew, afmt, as_)


@pytest.mark.parametrize("afmt,as_", base.ACTS)
@pytest.mark.parametrize("want,E,T,topk,N,H,spare,skew", CASES, ids=IDS)
def test_gated_backward(want, E, T, topk, N, H, spare, skew, afmt, as_):
    assert form(2, E, N // 2, 2 * H, T * topk) == want
    base.test_gated_backward(E, T, topk, H, N // 2, spare, skew, afmt, as_)


def test_the_few_row_form_is_aimed_at_elsewhere():
    """The small cases of the products' own tests are few-row calls."""
    for E, T, topk, H, Fc, *_ in base.GATED[:3]:
        assert form(1, E, Fc, 2 * H, T * topk) == ROWS
