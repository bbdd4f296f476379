"""Row counts whose blocks pass 2^32 threads: the token codes and the norms over a repeated
pattern of rows, every row with the bits of a small call."""
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
