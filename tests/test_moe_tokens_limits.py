"""Which rows of the few-token MoE layer fit into LDS: the documented sum, on
both sides of it (no GPU needed: the workspace is checked after the size)."""
import ctypes
import os

import pytest

from test_abi_host import _no_gpu_visible, pkg  # noqa: F401  (fixture)

pytestmark = pytest.mark.skipif(not _no_gpu_visible(), reason="placeholder pointers")
P = 0x1000


def status(lib, m, fmt, H, group, T, topk, E=1, F=64):
    w = m.fq_stored_w(fmt, group, P, P, P, P, P)
    d = m.fq_stored_w(m.FMT_NVFP4, 16, P, P, P, P, P)
    return lib.fq_moe_tokens(P, T, H, F, P, P, topk, 0, E, ctypes.byref(w), ctypes.byref(d), None,
                             None, P, P, 0, None)


def up(v, m):
    return -(-v // m) * m


def documented(H, group, T, topk):
    return 32 * (up(4 * (H // group), 8) + 8) + 2 * up(H, 64) + 16 + up(2 * T * topk, 16) + 11884


@pytest.mark.parametrize("T,topk", [(1, 1), (12, 8), (128, 8), (128, 64)])
@pytest.mark.parametrize("group", [16, 32, 48])
def test_small_groups_fit_as_documented(pkg, group, T, topk):  # noqa: F811
    """Whole rows (H a multiple of 64) and rows that end inside a chunk alike."""
    lib, seen = pkg.lib(), set()
    for fmt in (pkg.FMT_INT8, pkg.FMT_FP8_E4M3):
        for H in range(up(4096, group), 16385, group):
            fits = documented(H, group, T, topk) <= 163840
            want = pkg.FQ_ERR_WORKSPACE_TOO_SMALL if fits else pkg.FQ_ERR_UNSUPPORTED
            assert status(lib, pkg, fmt, H, group, T, topk) == want, (fmt, H, fits)
            seen.add((fits, H % 64 == 0))
    assert seen == ({(f, w) for f in (True, False) for w in (True, False)} if group == 16 else
                    {(True, True), (True, False)})


def test_the_named_sizes(pkg):  # noqa: F811
    lib, small, no = pkg.lib(), pkg.FQ_ERR_WORKSPACE_TOO_SMALL, pkg.FQ_ERR_UNSUPPORTED
    for H, T, topk, want in ((15136, 12, 8, small), (15152, 12, 8, no), (13504, 128, 64, small),
                             (13520, 128, 64, no), (8400, 128, 8, small), (8448, 128, 8, small)):
        assert status(lib, pkg, pkg.FMT_INT8, H, 16, T, topk) == want, H


@pytest.mark.parametrize("group", [32, 64, 96, 128])
def test_int4_groups_always_fit(pkg, group):  # noqa: F811
    for H in range(group, 16385, group):
        assert status(pkg.lib(), pkg, pkg.FMT_INT4, H, group, 128, 64) == \
            pkg.FQ_ERR_WORKSPACE_TOO_SMALL, H


def test_other_scale_modes_always_fit(pkg):  # noqa: F811
    for fmt, group in ((pkg.FMT_NVFP4, 16), (pkg.FMT_NONE, 0), (pkg.FMT_INT8, pkg.FQ_GROUP_TENSOR),
                       (pkg.FMT_INT8, None), (pkg.FMT_INT4, None)):
        for H in list(range(16, 2064, 16)) + list(range(14000, 16385, 16)):
            assert status(pkg.lib(), pkg, fmt, H, H if group is None else group, 128, 64) == \
                pkg.FQ_ERR_WORKSPACE_TOO_SMALL, H


def test_the_rule_for_channel_groups(repo_root):
    """test_gpu_moe_tokens_forms chooses its sizes by a copy of the launch's rule:
    whoever changes one changes the other."""
    src = os.path.join(repo_root, "moe_fake_quant_amd", "csrc", "moe_tokens.hip")
    with open(src) as f:
        text = f.read()
    for line in ("const int slots = a.P < a.E ? a.P : a.E;", "int mt = 4;",
                 "while (mt > 1 && (long)slots * ((a.agroups + mt - 1) / mt) < 1024) mt /= 2;",
                 "while (mt > 1 && 2 * mt * kTile * per_row > (20 << 10)) mt /= 2;"):
        assert text.count(line) == 1, line
