"""Element counts at the ends of the elementwise passes' ranges (host checks; what passes them
fails at the launch, without a device)."""
import pytest

from test_abi_host import host_only, pkg  # noqa: F401

P = 1 << 12      # an aligned placeholder address
INVALID, HIP = 1, 4


@host_only
@pytest.mark.parametrize("rows,want", [((3 << 33) // 2048, HIP), ((3 << 33) // 2048 + 1, INVALID),
                                       ((1 << 35) // 2048 - 1, INVALID)])
def test_vectors_of_eight_stay_in_32_bits(pkg, rows, want):  # noqa: F811
    """A grid of 2^30 threads steps over vectors of 8 elements by 32-bit indices, which
    wrap (and never end) beyond 3 * 2^30 vectors."""
    L, n = pkg.lib(), 2048
    assert L.fq_actfq(P, rows, n, None, P, None) == want
    assert L.fq_moe_gather_actfq(P, rows, n, P, 8, None, P, None) == want
    assert L.fq_swiglu_actfq(P, rows, P, n, None, None, P, None) == want
    assert L.fq_moe_combine_bwd(P, P, P, rows, 8, n, P, None) == want


@host_only
def test_vectors_of_sixteen_reach_further(pkg):  # noqa: F811
    L, n = pkg.lib(), 2048
    for rows, want in (((1 << 35) // n - 1, HIP), ((1 << 35) // n, INVALID)):
        assert L.fq_moe_combine(P, P, P, rows, 8, n, P, None) == want
        assert L.fq_moe_unpermute_reduce(P, P, None, rows, 8, n, None, P, None, None, 0, None) == want
        assert L.fq_swiglu_bwd(P, P, rows, P, n, None, P, None, None, 0, None) == want
