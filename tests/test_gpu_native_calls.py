"""The native marshalling of the int8, gated and norm calls: what it takes and refuses."""
import sys
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None


def z(*shape, t=torch.bfloat16):
    return torch.zeros(*shape, dtype=t, device="cuda")


def test_elements_of_another_type_are_refused():
    """Elements of the right size alone are not enough: float16 for bf16, integers for
    float32, float32 for int32, bool for codes."""
    x, codes, s, seg = z(4, 32), z(4, 32, t=torch.uint8), z(4, t=torch.float32), z(2, t=torch.int32)
    w, perm, half, y = z(1, 32, 32), z(4, t=torch.int32), z(4, 32, t=torch.float16), z(4, 32)
    st = F.StoredW(F.FMT_INT8, 32, z(1, 32, 32, t=torch.uint8), z(1, 32, t=torch.float32))
    h16, act = half[:, :16].contiguous(), F.ActQ(F.FMT_FP8_E4M3, z(1, t=torch.int32))
    gated = (x, 4, perm, 1, 4, seg, (1, 32, 32), w, None)
    bad = [lambda: F.fq_quantize_tokens(half, 4, 32, None, codes, s),
           lambda: F.fq_quantize_tokens(x, 4, 32, s[:1], codes, s),
           lambda: F.fq_quantize_tokens(x, 4, 32, None, codes.bool(), s),
           lambda: F.fq_quantize_tokens(x, 4, 32, None, codes, perm),
           lambda: F.fq_grouped_gemm_int8(codes, perm, 4, None, 1, 4, seg, (1, 32, 32), st, y),
           lambda: F.fq_grouped_gemm_int8(codes, s, 4, s, 1, 4, seg, (1, 32, 32), st, y),
           lambda: F.fq_grouped_gemm_int8(codes, s, 4, None, 1, 4, seg.float(), (1, 32, 32), st, y),
           lambda: F.fq_grouped_gemm_int8(codes, s, 4, None, 1, 4, seg, (1, 32, 32), st, half),
           lambda: F.fq_grouped_gemm_int8(codes, s, 4, None, 1, 4, seg, (1, 32, 32),
                                          F.StoredW(F.FMT_INT8, 32, st.codes, st.scale.int()), y),
           lambda: F.fq_grouped_gated_fwd(*gated, h16),
           lambda: F.fq_grouped_gated_fwd(half, *gated[1:], z(4, 16)),
           lambda: F.fq_grouped_gated_fwd(*gated[:-1], act, z(4, 16)),
           lambda: F.fq_grouped_gated_bwd(h16, *gated, y),
           lambda: F.fq_norm_residual_fwd(half, None, None, 1.0, None, z(32), 1e-6, 4, 32, None, y),
           lambda: F.fq_norm_residual_fwd(x, x, perm, 1.0, None, None, 1e-6, 4, 32, y),
           lambda: F.fq_norm_residual_bwd(x, None, None, None, None, 1.0, None, None, 1e-6, 4, 32, half)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="elements is wanted"):
            call()
            print("accepted:", i)
    # raw storage and signed codes are the same bytes
    F.fq_quantize_tokens(x.view(torch.int16), 4, 32, None, codes.view(torch.int8), s)
    F.fq_grouped_gemm_int8(codes.view(torch.int8), s, 4, perm, 1, 4, seg, (1, 32, 32), st, y.view(torch.int16))


def test_calls_release_the_interpreter_lock():
    """A thread that waits for the lock gets it during a call: the interpreter itself would
    not pass it on within 1000 s here."""
    woken, old = threading.Event(), sys.getswitchinterval()

    def waiter():
        time.sleep(0.1)       # without the lock; then waits for it
        woken.set()

    t = threading.Thread(target=waiter)
    try:
        sys.setswitchinterval(1000.0)
        t.start()
        end = time.monotonic() + 5.0
        while not woken.is_set() and time.monotonic() < end:
            F.fq_quantize_tokens(None, 0, 16, None, None, None)
        assert woken.is_set()
    finally:
        sys.setswitchinterval(old)
        t.join()
