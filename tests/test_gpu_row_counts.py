"""Row counts whose blocks pass 2^32 threads: token codes, norms, distillation and observed
groups over a repeated pattern of rows, every row with the bits of a small call."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_fake_quant_amd as F
else:  # collected on CPU only to be deselected by -m "not gpu"
    F = None

P = 61              # rows of the pattern
EPS = 1e-6
# rows of one wave (four to a block of 256 threads), rows of a block of 256
CASES = [((1 << 26) + 3 * P, 16), ((1 << 24) + 3 * P, 1040), ((1 << 24) + 3 * P, 528)]


def pattern(K, seed, rows):
    g = torch.Generator("cuda").manual_seed(seed)
    p = torch.randn(P, K, device="cuda", generator=g).bfloat16()
    return p, p.repeat(-(-rows // P), 1)[:rows]


def repeats(big, small):
    """Every row of `big` is the pattern's."""
    assert torch.equal(big[:P].view(torch.uint8), small.view(torch.uint8))
    step = 1 << 22
    for r in range(P, len(big), step):
        b = big[r:r + step]
        assert torch.equal(b.view(torch.uint8), big[r - P:r - P + len(b)].view(torch.uint8)), r


@pytest.mark.parametrize("rows,K", CASES[:2])
def test_token_codes_of_many_rows(rows, K):
    print(f"[many rows] codes {rows}x{K}", flush=True)
    p, x = pattern(K, 1, rows)
    e = lambda *s, t: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    c, s, c1, s1 = e(rows, K, t=torch.uint8), e(rows, t=torch.float32), e(P, K, t=torch.uint8), \
        e(P, t=torch.float32)
    F.fq_quantize_tokens(p, P, K, None, c1, s1)
    F.fq_quantize_tokens(x, rows, K, None, c, s)
    repeats(c, c1)
    repeats(s, s1)
    c.fill_(0xA5)
    live = torch.tensor([rows - 7], dtype=torch.int32, device="cuda")
    F.fq_quantize_tokens(x, rows, K, live, c, s)
    repeats(c[:-7], c1)
    assert bool((c[-7:] == 0xA5).all())


@pytest.mark.parametrize("T,H", [CASES[0], CASES[2]])
def test_norms_of_many_rows(T, H):
    print(f"[many rows] norms {T}x{H}", flush=True)
    p, x = pattern(H, 2, T)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    n, n1 = torch.empty_like(x), torch.empty_like(p)
    F.fq_norm_residual_fwd(p, None, None, 1.0, None, w, EPS, P, H, None, n1)
    F.fq_norm_residual_fwd(x, None, None, 1.0, None, w, EPS, T, H, None, n)
    repeats(n, n1)
    # the norm's rows as its gradients, and dx over them
    d1 = n1.clone()
    F.fq_norm_residual_bwd(None, n1, p, None, None, 1.0, None, w, EPS, P, H, dx=d1)
    F.fq_norm_residual_bwd(None, n, x, None, None, 1.0, None, w, EPS, T, H, dx=n)
    repeats(n, d1)


def test_distillation_of_many_rows():
    """2^23 rows of 512 threads each."""
    T, V, K = (1 << 23) + 3 * P, 16, 3
    print(f"[many rows] top-K KL {T}x{V}", flush=True)
    (ps, s), (pt, t) = pattern(V, 3, T), pattern(V, 4, T)
    e = lambda *d, t=torch.float32: torch.empty(*d, dtype=t, device="cuda")  # noqa: E731
    ws = e(256, t=torch.uint8)

    def run(s, t, n):
        idx, grad, tok, mean = e(n, K, t=torch.int32), e(n, K), e(n), e(1)
        F.fq_topk_kl(s, t, n, V, K, False, None, idx, grad, tok, mean, ws)
        return idx, grad, tok, float(mean)

    (i1, g1, l1, m1), (idx, grad, tok, mean) = run(ps, pt, P), run(s, t, T)
    repeats(idx, i1)
    repeats(tok, l1)
    repeats(grad, grad[:P])
    # one division by the number of rows apart
    assert torch.allclose(grad[:P] * T, g1 * P, rtol=2.0 ** -21, atol=0)
    # T is not a whole number of patterns: the mean of its rows, within 2^-11 of their sum of
    # magnitudes (2^13 terms a thread, then a tree)
    whole, rest = divmod(T, P)
    want = float((l1.double().sum() * whole + l1[:rest].double().sum()) / T)
    assert abs(mean - want) <= 2.0 ** -10 * float(l1.abs().mean())


def test_observed_groups_of_many_rows():
    """2^24 groups of 48 elements, a block of 256 threads each."""
    N, K = (1 << 24) + 3 * P, 48
    print(f"[many rows] observer {N}x{K}", flush=True)
    p, w = pattern(K, 5, N)
    s, s1, z, z1 = (torch.empty(n, device="cuda") for n in (N, P, N, P))
    for fmt in (F.FMT_INT8, F.FMT_INT4):
        zz = (z, z1) if fmt == F.FMT_INT4 else (None, None)
        F.observer_absmax_init(p, (1, P, K), fmt, K, 0, s1, zz[1])
        F.observer_absmax_init(w, (1, N, K), fmt, K, 0, s, zz[0])
        repeats(s, s1)
    repeats(z, z1)
