"""Newton-Schulz and the Muon step on matrices that lack directions (few tokens, repeated
rows, rows of zeros) and over long runs of steps.

In exact arithmetic every singular value follows x <- |x (a + b x^2 + c x^4)| from x_0 <= 1, so no result is
larger than that map's largest value, whatever the rank; `tops` follows it over a grid of
20001 points, whose spacing and the rounding of fp32 results are below the 10^-3 that each step's bound
is widened by.  A direction that U lacks is 0, or fp32's rounding of U grown up to the same bound.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_muon import MUON, U, iterate

pytestmark = pytest.mark.gpu
QUINTIC, CUBIC, LOGISTIC = (2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (2.5, -2.5, 0.0)

# one to four blocks of 16 rows a side in one launch and in two, wide and tall; planes
SHAPES = [(1, 8, 60), (2, 8, 768), (1, 700, 5), (2, 16, 40), (1, 2, 9), (2, 30, 64), (1, 300, 32), (2, 48, 200), (1, 770, 40),
          (2, 60, 200), (1, 200, 64), (1, 96, 200), (2, 150, 130)]


def tops(coeffs, steps):
    a, b, c = coeffs
    top = [1.0]
    for _ in range(steps):
        x = torch.linspace(0, top[-1], 20001, dtype=torch.float64)
        top.append(float((x * (a + b * x**2 + c * x**4)).abs().max()) * (1 + 1e-3))
    return top


def lacking(kind, B, M, N, g):
    """[B, M, N] of rank 1, 3 or m - 1, with rows (of the shorter side) repeated, of zeros, or of small integers."""
    m, n = min(M, N), max(M, N)

    def low(r):
        return torch.randn(B, m, r, generator=g) @ torch.randn(B, r, n, generator=g)

    if kind == "repeated":
        G = torch.randn(B, (m + 1) // 2, n, generator=g).repeat(1, 2, 1)[:, :m]
    elif kind == "zeros":
        G = torch.randn(B, m, n, generator=g)
        G[:, m // 3 + 1:] = 0
    elif kind == "integers":       # exact products: the missing directions are exactly zero
        G = (torch.randint(-3, 4, (B, m, 2), generator=g) @ torch.randint(-3, 4, (B, 2, n), generator=g)).float()
        G[:, 0, 0] += 1
    else:
        G = low({"rank1": 1, "rank3": min(3, m), "last": max(1, m - 1)}[kind])
    G = G * 1e-2
    return (G if M <= N else G.transpose(1, 2)).contiguous()


@pytest.mark.parametrize("kind", ["rank1", "rank3", "last", "repeated", "zeros", "integers"])
@pytest.mark.parametrize("B,M,N", SHAPES)
def test_long_runs_stay_bounded(B, M, N, kind):
    G = lacking(kind, B, M, N, torch.Generator().manual_seed(M + N)).cuda()
    for coeffs in (MUON, QUINTIC, CUBIC, LOGISTIC):
        top = tops(coeffs, 64)
        for steps in (5, 7, 8, 12, 16, 20, 24, 40, 64):
            say(f"newton_schulz {B}x{M}x{N} {kind} {coeffs} steps{steps}")
            out = gg.newton_schulz(G, steps=steps, coeffs=coeffs).double().cpu()
            assert torch.isfinite(out).all(), (coeffs, steps)
            s = float(torch.linalg.svdvals(out).max())
            assert s <= top[steps], f"{coeffs} steps{steps}: singular value {s} over {top[steps]}"


@pytest.mark.parametrize("B,M,N", [(2, 8, 768), (1, 16, 40), (1, 700, 5), (2, 30, 64), (1, 300, 32), (1, 48, 200), (1, 770, 40),
                                   (1, 60, 200), (1, 200, 64)])
def test_long_runs_against_64_bits(B, M, N):
    """Singular values of a 20th to all of the largest.  What a long run adds to the squares, 2^-46, is at most
    2^-46 / x^2 of a singular value x >= x_0 in each step, and steps of CUBIC and QUINTIC, which converge, do not multiply
    relative errors (|x f' / f| <= 1 on [0, 1]); those of MUON do by less than 3 (x up to 1.2), for each step
    taken.  fp64 itself: 64 terms, 17 products and 64 steps, 2^-33.  Then fp32's half step."""
    g = torch.Generator().manual_seed(M * N)
    m, n = min(M, N), max(M, N)
    left = torch.linalg.qr(torch.randn(B, m, m, generator=g, dtype=torch.float64)).Q
    right = torch.linalg.qr(torch.randn(B, n, m, generator=g, dtype=torch.float64)).Q.transpose(1, 2)
    s = torch.linspace(0.05, 1, m, dtype=torch.float64)
    G = (left * s @ right).float()
    G = (G if M <= N else G.transpose(1, 2)).contiguous()
    x0 = float(s[0] / s.norm()) * (1 - 1e-3)
    for coeffs, runs, grows in ((CUBIC, (34, 50, 64), 1), (QUINTIC, (20, 40, 64), 1), (MUON, (8, 9, 10), 3)):
        for steps in runs:
            say(f"newton_schulz {B}x{M}x{N} {coeffs} steps{steps}")
            got = gg.newton_schulz(G.cuda(), steps=steps, coeffs=coeffs).double().cpu()
            want = iterate(G, steps, coeffs, 1e-7, torch.float64)
            most = steps * 2.0**-46 / x0**2 * grows**steps + 2.0**-33
            off = (got - want).abs() - U * want.abs() * 1.001
            # an entry is at most the largest singular value's error: 1.2 bounds the values
            assert float(off.max()) <= 1.2 * most, f"{coeffs} steps{steps}: {float(off.max()):.3e} of {1.2 * most:.3e}"


def test_muon_step_of_few_tokens_over_long_runs():
    """Weights after steps of 24 and 64: finite, moved by at most the rate times the map's bound."""
    for B, M, N in SHAPES:
        g = torch.Generator().manual_seed(N)
        dW = lacking("rank3", B, M, N, g).cuda()
        for steps in (24, 64):
            W, mom = torch.zeros_like(dW), torch.zeros_like(dW)
            say(f"muon_step {B}x{M}x{N} rank 3 steps{steps}")
            gg.muon_step(W, dW, mom, 1.0, scale=1.0, steps=steps)
            out = W.double().cpu()
            assert torch.isfinite(out).all()
            assert float(torch.linalg.svdvals(out).max()) <= tops(MUON, steps)[steps]


def test_a_matrix_by_itself_and_in_a_batch_over_long_runs():
    """Zero, infinite and NaN matrices beside others, and the same bits alone, in long runs too."""
    for M, N in ((8, 60), (16, 500), (30, 64), (48, 100), (60, 200)):
        G = lacking("rank3", 5, M, N, torch.Generator().manual_seed(3))
        G[1] = 0
        G[2, 3, 5] = float("nan")
        G[3, M - 1, N - 1] = float("inf")
        say(f"newton_schulz {M}x{N} zero, nan, inf in a batch, 40 steps")
        out = gg.newton_schulz(G.cuda(), steps=40).cpu()
        assert (out[1] == 0).all() and torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
        for k in (0, 4):
            assert torch.equal(gg.newton_schulz(G[k].contiguous().cuda(), steps=40).cpu(), out[k])


@pytest.mark.parametrize("kind", ["rank1", "rank3", "last", "repeated", "zeros", "integers"])
@pytest.mark.parametrize("B,M,N", [c for c in SHAPES if min(c[1:]) <= 64])
def test_lacking_matrices_against_64_bits(B, M, N, kind):
    """Short runs, entry by entry, where each side still has fp64's rounding alone.  A, a sum of products of a side of up
    to 64, is off by 64 2^-53 between the directions that U has and lacks, and a step multiplies that by a (P is a on
    the one side, about 1 on the other).  The product of the polynomials, a^k in the directions that U lacks, takes it in by
    b A: 64 2^-53 |b| a^(2 (steps - 1)) of the largest entry at most in the last step, most of the sum over the steps.
    The rest is 2^-33 as for any matrix of such a side, and fp32's half step."""
    G = lacking(kind, B, M, N, torch.Generator().manual_seed(M + N))
    for steps in (1, 5, 7):
        most = 2.0**-33 + 64 * 2.0**-53 * abs(MUON[1]) * MUON[0] ** (2 * (steps - 1))
        say(f"newton_schulz {B}x{M}x{N} {kind} steps{steps}")
        got = gg.newton_schulz(G.cuda(), steps=steps).double().cpu()
        want = iterate(G, steps, MUON, 1e-7, torch.float64)
        off = (got - want).abs() - U * want.abs() * 1.001
        assert (off <= most * want.abs().amax((-1, -2), keepdim=True)).all(), float(off.max())


@pytest.mark.parametrize("kind", ["rank1", "rank3", "last", "repeated", "zeros", "integers"])
def test_steps_taken_together_stay_bounded(kind):
    """Muon steps in groups (long sides of 1.5 times the short and 128 tiles and more), over long runs."""
    for B, M, N in ((16, 256, 512), (40, 500, 200)):
        dW = lacking(kind, B, M, N, torch.Generator().manual_seed(N)).cuda()
        for coeffs in (MUON, QUINTIC, CUBIC, LOGISTIC):
            top = tops(coeffs, 64)
            for steps in (5, 12, 24, 64):
                W, mom = torch.zeros_like(dW), torch.zeros_like(dW)
                say(f"muon_step {B}x{M}x{N} {kind} {coeffs} steps{steps}")
                gg.muon_step(W, dW, mom, 1.0, scale=1.0, steps=steps, coeffs=coeffs)
                assert torch.isfinite(W).all(), (coeffs, steps)
                s = float(torch.linalg.svdvals(W[:2].double().cpu()).max())
                assert s <= top[steps], f"{coeffs} steps{steps}: singular value {s} over {top[steps]}"
