"""How near Newton-Schulz and the Muon step come to 64 bits, in units of fp32 arithmetic's own error on the same matrices.

Tolerance, in norms, so roundings count by their root mean square.  A value's pair of fp16 planes (2^-11 of 2^-11) is off
by 2^-24.6 of it, a product without that of its low parts by 2^-24.6, fp32's own rounding by 2^-25.3: a product of two pairs by
2.8 times that.  A sum of K products of either sign keeps sqrt(K) of theirs and adds K / sqrt(32) of its own (16 partial sums,
as torch's on a CPU), in fp32 and in the kernels alike.  The kernels' error over fp32's on the same matrix is then
sqrt((2.8^2 K + K^2 / 32) / (K + K^2 / 32)), 1.8 at K = 64 and less beyond; half as much again for chance: 3 times, plus
16 u |X| where fp32 happens to be nearly exact.

Steps taken together (Muon steps and bf16 results, long sides from 1.5 times the short on, 128 tiles and more of 128 x 128)
advance A = X X^T by itself, A <- P A P, for up to three steps, so that A's rounding grows by P^2 (a^2 = 11.9) a step where
that of X X^T does not.  The entry points promise 8 times the error of the iteration in fp32 for them.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_muon import BATCHES, MUON, U, gradient, iterate

pytestmark = pytest.mark.gpu


def norm(t):
    return t.double().square().sum((-1, -2)).sqrt()


@pytest.mark.parametrize("B,M,N", BATCHES + [(1, 300, 1000), (2, 192, 192), (1, 257, 2050)])
def test_batches_by_their_own_fp32_error(B, M, N):
    """Every tile of the products: the first, a middle and the last matrix of each batch, one step at a time."""
    g = torch.Generator(device="cuda").manual_seed(B + N)
    G = 1e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    G[:, : M // 8] *= 5
    some = sorted({0, B // 2, B - 1})
    for steps in (5, 4):
        say(f"newton_schulz {B}x{M}x{N} steps{steps}")
        out = gg.newton_schulz(G, steps=steps)[some].double().cpu()
        one = G[some].cpu()
        want = iterate(one, steps, MUON, 1e-7, torch.float64)
        f32 = iterate(one, steps, MUON, 1e-7, torch.float32)
        most = 3 * norm(f32 - want) + 16 * U * norm(want)
        assert (norm(out - want) <= most).all(), f"{(norm(out - want) / norm(want)).tolist()} of {(most / norm(want)).tolist()}"


@pytest.mark.parametrize("kind", ["noise", "low", "graded", "rank"])
@pytest.mark.parametrize("B,M,N", [(16, 256, 512), (16, 520, 256), (3, 512, 1500), (8, 768, 1536), (8, 1536, 768), (4, 1024, 4096),
                                   (40, 200, 500), (128, 70, 200), (300, 66, 100), (65, 200, 128), (33, 129, 300)])
def test_steps_taken_together(B, M, N, kind):
    """Noise, some strong directions over it, rows from 1 to 10^-4, and an eighth of the rank."""
    g = torch.Generator(device="cuda").manual_seed(M)
    dW = 1e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    if kind == "low":
        dW = gradient(B, M, N, 3).cuda()
    elif kind == "graded":
        dW *= torch.logspace(0, -4, M, device="cuda")[:, None]
    elif kind == "rank":
        r = min(M, N) // 8
        dW = dW[:, :, :r].contiguous() @ torch.randn(B, r, N, generator=g, device="cuda")
    for steps in (2, 3, 4, 5, 6, 7):
        W, mom = torch.zeros_like(dW), torch.zeros_like(dW)
        say(f"muon_step {B}x{M}x{N} {kind} steps{steps}")
        gg.muon_step(W, dW, mom, -1.0, beta=0.0, scale=1.0, steps=steps)
        torch.cuda.synchronize()
        want = iterate(dW, steps, MUON, 1e-7, torch.float64)
        f32 = iterate(dW, steps, MUON, 1e-7, torch.float32)
        # the batch as a whole: a single matrix's fp32 error may be small by chance
        off, unit, size = (float(norm(t).square().sum().sqrt()) for t in (W - want, f32 - want, want))
        assert off <= 8 * unit + 16 * U * size, f"steps{steps}: {off / unit} of the iteration in fp32, {off / size} of |X|"
