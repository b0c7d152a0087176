"""Newton-Schulz and the Muon step where eps holds X_0 = U / (|U| + eps) far below 1: a gradient, or the momentum
of an expert without tokens that decays, down to 10^-30 beside the default eps of 10^-7.

Tolerance, in norms, so roundings count by their root mean square.  A value's pair of fp16 planes (2^-11 of 2^-11) is off
by 2^-24.6 of it, a product without that of its low parts by 2^-24.6, fp32's own rounding by 2^-25.3: a product of two pairs by
2.8 times that.  A sum of K products of either sign keeps sqrt(K) of theirs and adds K / sqrt(32) of its own (16 partial sums,
as torch's on a CPU), in fp32 and in the kernels alike.  The kernels' error over fp32's on the same matrix is then
sqrt((2.8^2 K + K^2 / 32) / (K + K^2 / 32)), 1.8 at K = 64 and less beyond; half as much again for chance: 3 times, plus
16 u |X| where that happens to be nearly exact.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_muon import MUON, U, iterate

pytestmark = pytest.mark.gpu
CUBIC = (1.5, -0.5, 0.0)


def noise(B, M, N, size, seed):
    g = torch.Generator().manual_seed(seed)
    return size * torch.randn(B, M, N, generator=g)


def norm(t):
    return t.double().square().sum((-1, -2)).sqrt()


def check(got, G, steps, coeffs, eps, what, half=0.0):
    want = iterate(G, steps, coeffs, eps, torch.float64)
    f32 = iterate(G, steps, coeffs, eps, torch.float32).double()
    most = 3 * norm(f32 - want) + 16 * U * norm(want) + half * norm(want)
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    assert (norm(got - want) <= most).all(), f"{what}: {(norm(got - want) / norm(want)).tolist()} of {(most / norm(want)).tolist()}"


# tiles of 32, 64 and 128 rows; short sides on the fp64 path as well
@pytest.mark.parametrize("B,M,N", [(1, 100, 70), (2, 96, 160), (3, 130, 200), (1, 300, 600), (24, 260, 170), (80, 200, 200),
                                   (2, 20, 50), (1, 60, 200)])
@pytest.mark.parametrize("size", [1e-6, 1e-8, 1e-9, 1e-11, 1e-14, 1e-18, 1e-22, 1e-30])
def test_far_below_eps(B, M, N, size):
    G = noise(B, M, N, size, M)
    for dtype, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0**-8)):
        g = G.to(dtype)
        for steps, coeffs in ((1, MUON), (5, MUON), (6, CUBIC)):
            say(f"newton_schulz {B}x{M}x{N} {dtype} size {size} steps{steps} {coeffs}")
            check(gg.newton_schulz(g.cuda(), steps=steps, coeffs=coeffs), g, steps, coeffs, 1e-7, f"{dtype} {steps} {coeffs}", half)


@pytest.mark.parametrize("B,M,N", [(1, 100, 70), (3, 130, 200), (24, 260, 170)])
@pytest.mark.parametrize("size,steps", [(1e-9, 30), (1e-11, 40), (1e-14, 60), (1e-11, 25)])
def test_grown_from_far_below_eps(B, M, N, size, steps):
    """Enough steps of the converging iteration to bring singular values from rho to 1 (1.5^60 = 4 10^10), or on the way."""
    G = noise(B, M, N, size, N)
    say(f"newton_schulz {B}x{M}x{N} size {size} steps{steps}")
    check(gg.newton_schulz(G.cuda(), steps=steps, coeffs=CUBIC), G, steps, CUBIC, 1e-7, f"size {size}")


def test_matrices_of_a_batch_keep_their_own_scale():
    """Each as by itself: beside one far below eps, a zero one, an infinite one, one of 10^20."""
    for M, N in ((70, 100), (150, 90)):
        G = noise(6, M, N, 1e-3, 5)
        for k, by in enumerate((1e-20, 0.0, 1e23, 1e-9, 1.0, 1.0)):
            G[k] *= by
        G[5, 3, 4] = float("inf")
        say(f"newton_schulz {M}x{N} batch of magnitudes")
        out = gg.newton_schulz(G.cuda()).cpu()
        assert (out[1] == 0).all() and torch.isnan(out[5]).all()
        for k in (0, 2, 3, 4):
            assert torch.equal(gg.newton_schulz(G[k].contiguous().cuda()).cpu(), out[k])
            check(out[k:k + 1], G[k:k + 1], 5, MUON, 1e-7, f"matrix {k}")


@pytest.mark.parametrize("B,M,N", [(1, 70, 100), (16, 256, 512), (3, 512, 1500), (2, 30, 90)])
def test_momentum_that_decays(B, M, N):
    """A Muon step from the momentum alone, as an expert without tokens takes it: W moves by rate X, however small.
    Steps taken together (the two larger) multiply the rounding of A by P^2 in a group: the bound is 8 times fp32's."""
    mom0 = noise(B, M, N, 1e-13, N)
    for eps in (1e-7, 1e-3):
        W, mom = torch.zeros(B, M, N, device="cuda"), mom0.cuda()
        say(f"muon_step {B}x{M}x{N} decayed momentum eps {eps}")
        gg.muon_step(W, torch.zeros_like(W), mom, -1.0, beta=0.5, scale=1.0, nesterov=False, eps=eps)
        torch.cuda.synchronize()
        assert torch.equal(mom.cpu(), 0.5 * mom0)
        want = iterate(0.5 * mom0, 5, MUON, eps, torch.float64)
        f32 = iterate(0.5 * mom0, 5, MUON, eps, torch.float32).double()
        assert (norm(W.double().cpu() - want) <= 8 * norm(f32 - want) + 16 * U * norm(want)).all()
