"""The rule that chooses the form of an int8 or gated product, against measured times (host
only: without a device the rule counts 256 CUs, on which the times were taken)."""
import pytest

from test_abi_host import host_only, pkg  # noqa: F401

# us of one call in the forms few rows, 64 x 64, 128 x 128, 256 x 256 (None: not measured):
# (E, rows an expert, weight rows, contraction) -> int8, gated int8, gated bf16, its backward
TIMES = {
    (1, 16, 4096, 4096): ((7.8, 11.7, 16.6, 35.8), (9.2, 11.7, 16.7, 36.8), (14.8, 19.9, 30.2, 66.3),
                          (15.4, 19.8, 30.9, 68.9)),
    (1, 32, 4096, 4096): ((9.6, 11.5, 16.7, 35.7), (11.0, 11.7, 16.6, 36.6), (18.7, 20.0, 30.4, 67.2),
                          (19.4, 20.0, 31.2, 70.1)),
    (1, 48, 4096, 4096): ((12.5, 11.7, 16.8, 35.9), (14.5, 11.8, 17.0, 36.8), (25.6, 20.2, 30.6, 66.8),
                          (25.9, 20.4, 32.0, 69.5)),
    (1, 64, 4096, 4096): ((13.5, 11.7, 17.0, 36.1), (15.7, 11.8, 16.9, 36.9), (26.4, 20.8, 30.9, 67.3),
                          (27.4, 21.1, 32.3, 71.0)),
    (1, 128, 4096, 4096): ((23.9, 11.8, 17.7, 40.0), (15.8, 11.8, 17.9, 40.9), (26.6, 21.2, 35.7, 75.1),
                           (27.5, 21.4, 37.1, 78.8)),
    (1, 512, 4096, 4096): ((87, 17, 19, 44), (55, 17, 19, 46), (94, 30, 33, 81), (97, 31, 36, 86)),
    (1, 1024, 4096, 4096): ((None, 29, 22, 44), (None, 29, 21, 46), (None, 55, 37, 82), (None, 57, 40, 86)),
    (1, 2048, 4096, 4096): ((None, 55, 37, 50), (None, 54, 36, 49), (None, 107, 66, 83), (None, 117, 72, 86)),
    (1, 48, 2048, 2048): ((7.2, 7.9, 11.1, None), (8.7, 8.0, 11.2, None), (13.7, 11.7, 17.2, None),
                          (14.0, 11.7, 17.7, None)),
    (1, 64, 2048, 2048): ((7.8, 7.9, 11.2, None), (9.4, 7.9, 11.2, None), (14.6, 11.6, 17.2, None),
                          (15.0, 11.8, 17.7, None)),
    (1, 128, 2048, 2048): ((8.0, 8.0, 11.9, None), (9.4, 8.0, 12.1, None), (14.7, 11.8, 17.4, None),
                           (15.2, 12.0, 18.7, None)),
    (1, 64, 1024, 1024): ((4.9, 5.6, 7.9, None), (6.0, 5.6, 7.9, None), (8.5, 7.8, 11.4, None),
                          (8.9, 8.0, 12.0, None)),
    (4, 64, 1024, 1024): ((5.8, 6.8, 9.2, None), (6.8, 6.8, 9.2, None), (9.4, 8.6, 12.1, None),
                          (10.0, 8.9, 12.9, None)),
    (8, 64, 256, 512): ((4.0, 5.4, 7.3, None), (4.9, 5.4, 7.2, None), (5.9, 6.2, 8.9, None),
                        (6.4, 6.7, 9.7, None)),
    (1, 64, 1024, 4096): ((12.3, 11.6, 16.7, None), (14.6, 11.5, 16.8, None), (24.6, 19.0, 28.4, None),
                          (25.1, 18.8, 28.8, None)),
    (128, 16, 1536, 2048): ((121, 80, 86, 90), (131, 79, 83, 90), (211, 146, 155, 162), (227, 155, 158, 170)),
    (128, 64, 1536, 2048): ((None, 95, 94, 93), (None, 92, 89, 92), (None, 167, 164, 202),
                            (None, 178, 180, 214)),
    (128, 128, 1536, 2048): ((None, 143, 120, 104), (None, 140, 111, 98), (None, 249, 201, 200),
                             (None, 259, 233, 217)),
    (128, 256, 1536, 2048): ((None, 250, 190, 132), (None, 245, 175, 126), (None, 416, 273, 215),
                             (None, 443, 306, 237)),
    (64, 1024, 2048, 768): ((None, 298, 211, 154), (None, 279, 179, 143), (None, 411, 281, 216),
                            (None, 503, 366, 270)),
}


@host_only
@pytest.mark.parametrize("size", TIMES)
def test_the_rule_agrees_with_the_times(pkg, size):  # noqa: F811
    """The chosen form is within a tenth of the fastest, the spread of the times between cards."""
    E, per, N, K = size
    for name, times in zip(("int8", "gated int8", "gated", "backward"), TIMES[size]):
        kind = {"int8": 0, "backward": 2}.get(name, 1)
        form = pkg.lib().fq_internal_product_form(kind, E, N if kind == 0 else N // 2,
                                                  K * (1 if "int8" in name else 2), E * per)
        best = min(t for t in times if t is not None)
        assert times[form] is not None and times[form] <= 1.1 * best, (name, form, times)
