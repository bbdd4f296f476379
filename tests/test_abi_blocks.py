"""Refusals of the int8 products, the gated block and the norms: every call below is
rejected by the host checks before anything is enqueued, so the placeholder
addresses are never read (run where no GPU is visible)."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_abi_host import host_only, pkg  # noqa: F401

INVALID, UNSUPPORTED, WS = 1, 2, 3
P = 1 << 12      # an aligned placeholder address
NAN, INF = float("nan"), float("inf")


def call(pkg, name, args):  # noqa: F811
    st = getattr(pkg.lib(), name)(*args)
    return st, pkg.lib().fq_last_error().decode()


def stored(pkg, fmt=1, group=64, codes=P, scale=P):  # noqa: F811
    return ctypes.byref(pkg.fq_stored_w(fmt, group, codes, scale, None, None, None))


def int8_args(pkg, **kw):  # noqa: F811
    a = dict(x=P, sx=P, rows=8, perm=None, topk=1, R=8, seg=P, shape=(2, 32, 64), w=None, y=P)
    a.update(kw)
    return (a["x"], a["sx"], a["rows"], a["perm"], a["topk"], a["R"], a["seg"], pkg.fq_shape(*a["shape"]),
            a["w"] or stored(pkg), a["y"], None, 0, None)


INT8_BAD = [(dict(x=None), INVALID), (dict(sx=None), INVALID), (dict(seg=None), INVALID),
            (dict(y=None), INVALID), (dict(R=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=7), INVALID),
            (dict(perm=P, topk=0), INVALID), (dict(x=P + 8), INVALID), (dict(y=P + 2), INVALID),
            (dict(sx=P + 2), INVALID), (dict(shape=(0, 32, 64)), INVALID), (dict(shape=(2, 24, 64)), UNSUPPORTED),
            (dict(shape=(2, 32, 72)), UNSUPPORTED), (dict(shape=(1025, 32, 64)), UNSUPPORTED),
            (dict(shape=(1, 1 << 17, 1 << 15)), INVALID),
            (dict(perm=P, rows=1 << 27), UNSUPPORTED), (dict(shape=(1, 32, 1 << 21)), UNSUPPORTED)]


@host_only
@pytest.mark.parametrize("fn", ["fq_grouped_gemm_int8", "fq_grouped_gated_int8"])
@pytest.mark.parametrize("kw,status", INT8_BAD)
def test_int8_products_refuse(pkg, fn, kw, status):  # noqa: F811
    st, msg = call(pkg, fn, int8_args(pkg, **kw))
    assert st == status and msg


@host_only
@pytest.mark.parametrize("fn", ["fq_grouped_gemm_int8", "fq_grouped_gated_int8"])
def test_int8_products_refuse_other_weights(pkg, fn):  # noqa: F811
    for w, status in ((dict(fmt=3), UNSUPPORTED), (dict(fmt=0), UNSUPPORTED), (dict(group=16), UNSUPPORTED),
                      (dict(group=0), UNSUPPORTED), (dict(codes=None), INVALID), (dict(codes=P + 4), INVALID),
                      (dict(scale=None), INVALID), (dict(scale=P + 1), INVALID)):
        assert call(pkg, fn, int8_args(pkg, w=stored(pkg, **w)))[0] == status, w
    args = list(int8_args(pkg))
    args[8] = None
    assert call(pkg, fn, args)[0] == INVALID
    big = dict(shape=(1, 32, 131072), w=stored(pkg, group=131072))
    assert call(pkg, fn, int8_args(pkg, **big))[0] == UNSUPPORTED     # int32 sums
    assert call(pkg, fn, int8_args(pkg, R=0, x=None, sx=None, rows=0, y=None))[0] == 0


@host_only
def test_gated_product_needs_whole_halves(pkg):  # noqa: F811
    assert call(pkg, "fq_grouped_gated_int8", int8_args(pkg, shape=(2, 48, 64)))[0] == UNSUPPORTED
    assert call(pkg, "fq_grouped_gemm_int8", int8_args(pkg, shape=(2, 48, 64), R=0))[0] == 0


def gated_args(pkg, bwd, **kw):  # noqa: F811
    a = dict(daq=P, x=P, rows=8, perm=None, topk=1, R=8, seg=P, shape=(2, 64, 64), w=P, fmt=0, scale=None,
             out=P, aq=None)
    a.update(kw)
    q = ctypes.byref(pkg.fq_act_q(a["fmt"], a["scale"]))
    head = (a["x"], a["rows"], a["perm"], a["topk"], a["R"], a["seg"], pkg.fq_shape(*a["shape"]), a["w"], q,
            a["out"])
    return ((a["daq"],) + head + (a["aq"],) if bwd else head) + (None, 0, None)


GATED_BAD = [(dict(x=None), INVALID), (dict(seg=None), INVALID), (dict(out=None), INVALID),
             (dict(w=None), INVALID), (dict(w=P + 8), INVALID), (dict(x=P + 8), INVALID), (dict(R=-2), INVALID),
             (dict(rows=3), INVALID), (dict(perm=P, topk=-1), INVALID), (dict(fmt=2, scale=P), INVALID),
             (dict(fmt=3), INVALID), (dict(fmt=9, scale=P), INVALID), (dict(shape=(2, 16, 64)), UNSUPPORTED),
             (dict(shape=(2, 64, 8)), UNSUPPORTED), (dict(shape=(1025, 64, 64)), UNSUPPORTED),
             (dict(shape=(1, 1 << 16, 1 << 15)), UNSUPPORTED), (dict(perm=P, rows=1 << 26), UNSUPPORTED),
             (dict(shape=(1, 64, 1 << 21)), UNSUPPORTED)]


@host_only
@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", GATED_BAD)
def test_gated_block_refuses(pkg, bwd, kw, status):  # noqa: F811
    fn = "fq_grouped_gated_bwd" if bwd else "fq_grouped_gated_fwd"
    st, msg = call(pkg, fn, gated_args(pkg, bwd, **kw))
    assert st == status and msg


@host_only
def test_gated_backward_refuses_its_own(pkg):  # noqa: F811
    for kw in (dict(daq=None), dict(daq=P + 8), dict(aq=P + 4)):
        assert call(pkg, "fq_grouped_gated_bwd", gated_args(pkg, True, **kw))[0] == INVALID
    nothing = dict(R=0, rows=0, x=None, out=None, daq=None)
    for bwd in (False, True):
        fn = "fq_grouped_gated_bwd" if bwd else "fq_grouped_gated_fwd"
        assert call(pkg, fn, gated_args(pkg, bwd, **nothing))[0] == 0


@host_only
def test_quantize_tokens_refuses(pkg):  # noqa: F811
    for args, status in (((None, 4, 64, None, P, P), INVALID), ((P, 4, 64, None, None, P), INVALID),
                         ((P, 4, 64, None, P, None), INVALID), ((P, -1, 64, None, P, P), INVALID),
                         ((P, 4, 24, None, P, P), INVALID), ((P, 4, 0, None, P, P), INVALID),
                         ((P + 2, 4, 64, None, P, P), INVALID), ((P, 4, 64, None, P + 1, P), INVALID),
                         ((P, 4, 64, None, P, P + 2), INVALID),
                         ((P, 1 << 30, 64, None, P, P), INVALID), ((None, 0, 64, None, None, None), 0)):
        assert call(pkg, "fq_quantize_tokens", args + (None,))[0] == status, args


def norm_fwd(**kw):
    a = dict(x=P, b=P, gate=P, alpha=1.0, w_post=P, w_pre=P, eps=1e-6, T=4, H=64, y=P, n=P, codes=None,
             scale=None)
    a.update(kw)
    return tuple(a.values()) + (None,)


def norm_bwd(**kw):
    a = dict(dy=P, dn=P, y=P, b=P, gate=P, alpha=1.0, w_post=P, w_pre=P, eps=1e-6, T=4, H=64, dx=P, db=P,
             dgate=P, dw_post=None, dw_pre=None, ws=None, ws_bytes=0)
    a.update(kw)
    return tuple(a.values()) + (None,)


SHARED_BAD = [(dict(T=1 << 30), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=24), INVALID), (dict(H=16400), UNSUPPORTED),
              (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
              (dict(alpha=INF), INVALID), (dict(alpha=NAN), INVALID), (dict(b=None), INVALID),
              (dict(b=P + 8), INVALID), (dict(w_post=P + 2), INVALID), (dict(w_pre=P + 2), INVALID)]


@host_only
@pytest.mark.parametrize("kw,status", SHARED_BAD + [
    (dict(x=None), INVALID), (dict(y=None, n=None), INVALID), (dict(w_pre=None), INVALID),
    (dict(n=None), INVALID), (dict(codes=P), INVALID), (dict(scale=P), INVALID), (dict(x=P + 8), INVALID),
    (dict(y=P + 8), INVALID), (dict(codes=P + 4, scale=P), INVALID), (dict(codes=P, scale=P + 2), INVALID)])
def test_norm_forward_refuses(pkg, kw, status):  # noqa: F811
    st, msg = call(pkg, "fq_norm_residual_fwd", norm_fwd(**kw))
    assert st == status and msg


@host_only
@pytest.mark.parametrize("kw,status", SHARED_BAD + [
    (dict(dy=None, dn=None), INVALID), (dict(y=None), INVALID), (dict(w_pre=None), INVALID),
    (dict(dx=None, db=None, dgate=None), INVALID), (dict(dn=None, dw_pre=P), INVALID),
    (dict(w_post=None, dw_post=P), INVALID), (dict(gate=None), INVALID), (dict(dx=P + 8), INVALID),
    (dict(dw_pre=P), WS), (dict(dw_post=P, ws=P, ws_bytes=64), WS), (dict(dw_pre=P, ws=P + 8, ws_bytes=1 << 20), INVALID)])
def test_norm_backward_refuses(pkg, kw, status):  # noqa: F811
    st, msg = call(pkg, "fq_norm_residual_bwd", norm_bwd(**kw))
    assert st == status and msg


def test_workspace_sizes(pkg):  # noqa: F811
    ws = pkg.fq_workspace_bytes
    assert ws(pkg.FQ_OP_NORM, (1, 0, 64), 0, 0) == 0
    assert ws(pkg.FQ_OP_NORM, (1, 1, 64), 0, 0) >= 2 * 64 * 4
    assert ws(pkg.FQ_OP_NORM, (1, 1 << 20, 16384), 0, 0) < 1 << 27
    assert ws(pkg.FQ_OP_NORM, (1, -1, 64), 0, 0) == 0
    for op in (pkg.FQ_OP_GEMM_INT8, pkg.FQ_OP_GATED):
        assert ws(op, (4, 64, 64), 100, 0) == 0


def test_native_marshalling_checks_its_arguments(pkg):  # noqa: F811
    with pytest.raises(TypeError):
        pkg._b.fq_quantize_tokens(None, 0)


DIRECT = """
import ctypes
import moe_fake_quant_amd as pkg
P = 1 << 12
lib, sh = pkg.lib(), pkg.fq_shape(2, 64, 64)
w = ctypes.byref(pkg.fq_stored_w(1, 64, P, P, None, None, None))
for topk in (0, -1):
    for fn in ("fq_grouped_gemm_int8", "fq_grouped_gated_int8"):
        print(getattr(lib, fn)(P, P, 8, None, topk, 8, P, sh, w, P, None, 0, None))
    print(lib.fq_grouped_gated_fwd(P, 8, None, topk, 8, P, sh, P, None, P, None, 0, None))
    print(lib.fq_grouped_gated_bwd(P, P, 8, None, topk, 8, P, sh, P, None, P, None, None, 0, None))
"""


@host_only
def test_direct_rows_do_not_read_topk(pkg):  # noqa: F811
    """Without perm any topk passes the checks: the calls get as far as the launch, which
    fails here without a device (in a process of its own, which an arithmetic trap would end)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", DIRECT], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.split() == ["4"] * 8, r.stdout


@host_only
def test_norms_without_rows(pkg):  # noqa: F811
    """Empty tensors have no address: with T = 0 every row tensor may be NULL, and nothing is
    enqueued without the weights' gradients."""
    rows = dict(T=0, x=None, b=None, gate=None, y=None, n=None)
    for kw in (rows, dict(rows, w_post=None), dict(rows, w_pre=None), dict(rows, codes=P)):
        assert call(pkg, "fq_norm_residual_fwd", norm_fwd(**kw))[0] == 0, kw
    rows = dict(T=0, dy=None, dn=None, y=None, b=None, gate=None, dx=None, db=None, dgate=None)
    for kw in (rows, dict(rows, w_post=None), dict(rows, w_pre=None)):
        assert call(pkg, "fq_norm_residual_bwd", norm_bwd(**kw))[0] == 0, kw
    assert call(pkg, "fq_norm_residual_fwd", norm_fwd(T=0, H=24))[0] == INVALID


@host_only
def test_gated_backward_refuses_columns_past_its_offsets(pkg):  # noqa: F811
    """64 rows of dA are reached by 32-bit offsets: 128 F bytes, up to 2^32. (What passes
    the checks fails at the launch, without a device.)"""
    for F, bwd, fwd in ((1 << 25, 4, 4), ((1 << 25) + 16, UNSUPPORTED, 4)):
        assert call(pkg, "fq_grouped_gated_bwd", gated_args(pkg, True, shape=(1, 2 * F, 16)))[0] == bwd
        assert call(pkg, "fq_grouped_gated_fwd", gated_args(pkg, False, shape=(1, 2 * F, 16)))[0] == fwd


@host_only
def test_products_refuse_row_counts_at_the_end_of_int32(pkg):  # noqa: F811
    """Row counts are rounded up to tiles and experts in int32. (What passes the checks
    fails at the launch, without a device.)"""
    top = (1 << 31) - 1
    for R, want in ((top - 1024, 4), (top - 1023, UNSUPPORTED), (top, UNSUPPORTED)):
        kw = dict(R=R, rows=R, shape=(2, 32, 16))
        for fn in ("fq_grouped_gemm_int8", "fq_grouped_gated_int8"):
            assert call(pkg, fn, int8_args(pkg, w=stored(pkg, group=16), **kw))[0] == want, (fn, R)
        assert call(pkg, "fq_grouped_gated_fwd", gated_args(pkg, False, **kw))[0] == want, R
        assert call(pkg, "fq_grouped_gated_bwd", gated_args(pkg, True, **kw))[0] == want, R
