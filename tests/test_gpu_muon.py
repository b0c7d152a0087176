"""Newton-Schulz and the Muon step on the GPU against the iteration in 64 bits.

Tolerances.  A step multiplies an error in a small singular direction by
up to a, so how far fp32 ends from 64 bits depends on the matrix: it is taken
from the matrix itself, as the error of the same iteration in fp32 on the
CPU.  The kernels' operands hold 22 bits where fp32 has 24 and leave out
products of two low parts (2^-22), so each of their roundings is at most
2 * 4 = 8 of fp32's, and the bound on the Frobenius norm of the error is 8 times
that plus 16 u |X| where fp32 happens to be nearly exact (u = 2^-24).  Short sides
of at most 32, and 64 in few matrices, run in fp64: u |x| for the one rounding, and
2^-40 of the largest entry (beyond 32: 17 products of 64 terms, grown by a^5 = 485,
are 64 * 17 * 485 * 2^-53 < 2^-33).  bf16 results add half a step, 2^-8 of each entry.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
MUON = (3.4445, -4.7750, 2.0315)
SMALL = [(1, 1, 1), (2, 1, 5), (3, 32, 7), (1, 8, 768), (1, 768, 8), (2, 32, 300), (1, 31, 129), (1, 5, 4100),
         (2, 17, 17), (1, 4097, 3), (3, 16, 769), (2, 32, 256), (2, 257, 32), (1, 20, 9000), (2, 384, 16),
         (1, 385, 9), (2, 5, 384), (3, 9, 40)]
LARGE = [(1, 33, 33), (2, 40, 100), (1, 64, 64), (1, 65, 127), (1, 129, 128), (2, 200, 130), (1, 130, 200),
         (3, 128, 256), (1, 300, 1000), (1, 1000, 333), (2, 192, 192), (1, 257, 2050), (5, 768, 96),
         (2, 48, 300), (1, 64, 1000), (3, 700, 49), (1, 50, 20000), (1, 9000, 37), (4, 65, 65)]


# Batches that reach every tile of the products: 64 (split), 128 in one round and more, 256 (also with
# tiles that end past the padded matrix), and, for bf16, steps in groups (long sides of 1.5 times the short).
BATCHES = [(3, 500, 700), (6, 700, 500), (8, 256, 1024), (9, 600, 1300), (24, 520, 330), (150, 300, 300),
           (150, 180, 460), (16, 1024, 1024), (90, 256, 256), (17, 500, 1000), (1, 2100, 2100),
           (513, 48, 40), (257, 60, 64), (40, 1000, 64), (70, 48, 1100)]


def gradient(B, M, N, seed, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    r = max(1, min(M, N) // 16)
    low = torch.randn(B, M, r, generator=g) @ torch.randn(B, r, N, generator=g)
    return size * (low * (2 / r ** 0.5) + torch.randn(B, M, N, generator=g))


def iterate(G, steps, coeffs, eps, dt):
    a, b, c = coeffs
    tall = G.shape[-2] > G.shape[-1]
    X = G.to(dt)
    X = X.transpose(-1, -2) if tall else X
    X = X / (X.double().square().sum((-1, -2), keepdim=True).sqrt() + eps).to(dt)
    for _ in range(steps):
        A = X @ X.transpose(-1, -2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.transpose(-1, -2) if tall else X


def check(got, G, dtype, steps=5, coeffs=MUON, eps=1e-7, what=""):
    want = iterate(G, steps, coeffs, eps, torch.float64)
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    off = got - want
    if min(G.shape[-2:]) <= 64:
        most = U * want.abs() + 2.0 ** (-40 if min(G.shape[-2:]) <= 32 else -33) * want.abs().amax((-1, -2), keepdim=True)
        if dtype == torch.bfloat16:
            most = most + 2.0 ** -8 * want.abs()
        assert (off.abs() <= most * 1.001).all(), f"{what}: {float((off.abs() - most).max()):.3e} over"
        return
    f32 = iterate(G, steps, coeffs, eps, torch.float32).double()
    norm = lambda t: t.square().sum((-1, -2)).sqrt()  # noqa: E731
    most = 8 * norm(f32 - want) + 16 * U * norm(want)
    if dtype == torch.bfloat16:
        most = most + 2.0 ** -8 * norm(want)
    assert (norm(off) <= most).all(), f"{what}: {norm(off).tolist()} of {most.tolist()}"
    # no entry of a kind by itself (an edge, a corner) is wrong
    assert float(off.abs().max()) <= float(most.max()) * 0.5 + (2.0 ** -8 * float(want.abs().max()) if dtype == torch.bfloat16 else 0), what


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,M,N", SMALL + LARGE)
def test_newton_schulz(B, M, N, dtype):
    G = gradient(B, M, N, B + M + N).to(dtype)
    say(f"newton_schulz {B}x{M}x{N} {dtype}")
    out = gg.newton_schulz(G.cuda())
    torch.cuda.synchronize()
    check(out, G, dtype, what=f"{B}x{M}x{N}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,M,N", BATCHES)
def test_newton_schulz_batches(B, M, N, dtype):
    """The reference of all matrices in 64 bits on the GPU, and the fp32 error too."""
    g = torch.Generator(device="cuda").manual_seed(B + M)
    G = 1e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    G[:, : M // 8] *= 5
    G = G.to(dtype)
    for steps in (5, 4):
        say(f"newton_schulz {B}x{M}x{N} {dtype} steps{steps}")
        out = gg.newton_schulz(G, steps=steps).double()
        torch.cuda.synchronize()
        want = iterate(G, steps, MUON, 1e-7, torch.float64)
        f32 = iterate(G.cpu(), steps, MUON, 1e-7, torch.float32).double().cuda() if B * M * N < 3e6 else None
        norm = lambda t: t.square().sum((-1, -2)).sqrt()  # noqa: E731
        # where the fp32 run on the CPU takes too long: its error is at least 2 u |X| (X's last rounding and a product's)
        most = 8 * (norm(f32 - want) if f32 is not None else 30 * U * norm(want)) + 16 * U * norm(want)
        if dtype == torch.bfloat16:
            most = most + 2.0 ** -8 * norm(want)
        assert (norm(out - want) <= most).all(), f"{(norm(out - want) / norm(want)).max()}"
        worst = (out - want).abs().amax((-1, -2)) / want.abs().amax((-1, -2))
        assert float(worst.max()) < (2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0) + 1e-4


@pytest.mark.parametrize("B,M,N,dtype", [(16, 256, 512, torch.float32), (16, 520, 256, torch.bfloat16),
                                         (3, 512, 1500, torch.float32)])
def test_muon_step_batches(B, M, N, dtype):
    """Steps in groups (long sides of 1.5 times the short, enough tiles): the update against 64 bits."""
    lr, beta, scale = 0.02, 0.95, 1.3
    g = torch.Generator(device="cuda").manual_seed(M)
    W0 = (torch.randn(B, M, N, generator=g, device="cuda") / M ** 0.5).to(dtype)
    dW = 1e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    mom = 5e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    W = torch.zeros_like(W0)                  # the update alone, without W's own rounding above it
    say(f"muon_step {B}x{M}x{N} {dtype}")
    m0 = mom.clone()
    gg.muon_step(W, dW, mom, lr, beta=beta, scale=scale)
    torch.cuda.synchronize()
    f = lambda v: torch.tensor(v, dtype=torch.float32).double().item()  # noqa: E731
    u = dW.double() + f(beta) * mom.double()
    X = iterate(u, 5, MUON, 1e-7, torch.float64)
    x32 = iterate(u[:2].float().cpu(), 5, MUON, 1e-7, torch.float32).double().cuda()
    off = 8 * (x32 - X[:2]).square().mean().sqrt() + 16 * U * X.square().mean().sqrt()
    want = -f(lr) * f(scale) * X
    rms = (W.double() - want).square().mean().sqrt()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert rms <= lr * scale * off + (half + 4 * U) * want.square().mean().sqrt()
    W = W0.clone()
    gg.muon_step(W, dW, m0, lr, beta=beta, scale=scale)
    assert torch.equal(m0, mom)
    assert ((W.double() - (W0.double() + want)).abs() <= half * (W0.double() + want).abs() * 1.01 + 4 * U * W0.double().abs()
            + 1e-4 * want.abs().max()).all()


@pytest.mark.parametrize("M,N", [(24, 90), (90, 24), (96, 160), (160, 96), (40, 90), (160, 60)])
@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, MUON), (6, MUON), (7, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5)),
                                          (2, (0.0, 0.0, 0.0)), (4, (1e-3, 0.0, 0.0)), (10, (0.1, 0.0, 0.0)),
                                          (2, (0.0, 0.1, 0.0))])
def test_steps_and_coefficients(M, N, steps, coeffs):
    G = gradient(2, M, N, 77)
    say(f"newton_schulz {M}x{N} steps{steps} {coeffs}")
    out = gg.newton_schulz(G.cuda(), steps=steps, coeffs=coeffs)
    torch.cuda.synchronize()
    check(out, G, torch.float32, steps, coeffs, what=f"{steps} {coeffs}")


@pytest.mark.parametrize("M,N", [(20, 50), (100, 70), (40, 64)])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e25])
def test_magnitudes(M, N, size):
    """The norm and the planes hold gradients of any magnitude (eps far below their norm)."""
    G = gradient(1, M, N, 5, size)
    say(f"newton_schulz {M}x{N} size {size}")
    out = gg.newton_schulz(G.cuda(), eps=1e-36)
    torch.cuda.synchronize()
    check(out, G, torch.float32, eps=1e-36, what=f"size {size}")


@pytest.mark.parametrize("M,N,r", [(96, 200, 5), (200, 96, 5), (150, 150, 20), (30, 64, 3), (64, 64, 1)])
def test_rank_deficient(M, N, r):
    """A gradient of fewer tokens than the width: the directions it lacks stay near zero."""
    g = torch.Generator().manual_seed(r)
    G = (torch.randn(M, r, generator=g) @ torch.randn(r, N, generator=g))[None] * 1e-2
    say(f"newton_schulz {M}x{N} rank {r}")
    out = gg.newton_schulz(G.cuda())
    torch.cuda.synchronize()
    s = torch.linalg.svdvals(out[0].double().cpu())
    assert float(s[:r].max()) < 1.25 and float(s[:r].min()) > 0.3
    # what fp32 rounding leaves in the missing directions, 16 u of the norm, times a^5 = 485
    assert r >= min(M, N) or float(s[r:].max()) < 16 * U * r ** 0.5 * 485
    if min(M, N) > 32:
        check(out, G, torch.float32, what=f"rank {r}")


@pytest.mark.parametrize("M,N", [(16, 40), (70, 90), (90, 70), (50, 200)])
def test_zero_infinite_and_nan_matrices(M, N):
    G = gradient(5, M, N, 9)
    G[1] = 0
    G[2, 3, 5] = float("nan")
    G[3, M - 1, N - 1] = float("inf")
    say(f"newton_schulz {M}x{N} zero, nan, inf in a batch")
    out = gg.newton_schulz(G.cuda()).cpu()
    assert (out[1] == 0).all()
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    for k in (0, 4):
        check(out[k:k + 1], G[k:k + 1], torch.float32, what=f"matrix {k}")
        assert torch.equal(gg.newton_schulz(G[k].contiguous().cuda()).cpu(), out[k])     # the batch changes nothing


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype,copy", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("B,M,N", [(1, 1, 3), (2, 8, 70), (2, 70, 8), (2, 100, 150), (3, 150, 100), (1, 130, 131),
                                   (2, 768, 8), (3, 13, 500), (1, 300, 20), (2, 31, 600), (1, 384, 16),
                                   (2, 45, 200), (1, 300, 64)])
def test_muon_step(B, M, N, dtype, copy, nesterov):
    lr, beta, decay, scale = 0.02, 0.9, 0.1, 1.4
    g = torch.Generator().manual_seed(M * N)
    W0 = (torch.randn(B, M, N, generator=g) / M ** 0.5).to(dtype)
    dW, m0 = gradient(B, M, N, 1), gradient(B, M, N, 2, 1e-2)
    W, mom = W0.cuda(), m0.cuda()
    Wc = torch.empty(B, M, N, dtype=torch.bfloat16, device="cuda") if copy else None
    say(f"muon_step {B}x{M}x{N} {dtype} copy{copy} nesterov{nesterov}")
    assert gg.muon_step(W, dW.cuda(), mom, lr, beta=beta, weight_decay=decay, scale=scale, nesterov=nesterov,
                        W_bf16=Wc) is W
    torch.cuda.synchronize()
    f = lambda v: torch.tensor(v, dtype=torch.float32).double()  # noqa: E731
    m = f(beta) * m0.double() + dW.double()
    assert ((mom.double().cpu() - m).abs() <= U * m.abs() * 1.001).all()
    u = dW.double() + f(beta) * mom.double().cpu() if nesterov else mom.double().cpu()
    X = iterate(u, 5, MUON, 1e-7, torch.float64)
    # fp32's own error from the rounded U, per entry as a share of the matrix's largest
    xoff = (iterate(u.float(), 5, MUON, 1e-7, torch.float32).double() - X).square().sum((-1, -2), keepdim=True).sqrt()
    want = (1 - f(lr) * f(decay)) * W0.double() - f(lr) * f(scale) * X
    most = 4 * U * (W0.double().abs() + lr * scale * X.abs()) + lr * scale * (8 * xoff + 16 * U * X.abs().amax((-1, -2), keepdim=True))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert ((W.double().cpu() - want).abs() <= most + half * want.abs() * 1.01).all()
    if copy:
        assert torch.equal(Wc, W.to(torch.bfloat16))


def test_default_scale():
    W, g = torch.zeros(64, 256, device="cuda"), gradient(1, 64, 256, 4)[0].cuda()
    say("muon_step default scale")
    gg.muon_step(W, g, torch.zeros_like(g), 1.0, beta=0.0)
    X = gg.newton_schulz(g)
    assert torch.allclose(W, -2.0 * X, rtol=1e-6, atol=0)
    W2, g2 = torch.zeros(256, 64, device="cuda"), g.t().contiguous()
    gg.muon_step(W2, g2, torch.zeros_like(g2), 1.0, beta=0.0)
    assert torch.allclose(W2, -gg.newton_schulz(g2), rtol=1e-6, atol=0)


def test_in_place_empty_and_repeated():
    for M, N in ((20, 60), (90, 140)):
        G = gradient(2, M, N, 3).cuda()
        say(f"newton_schulz {M}x{N} in place")
        want = gg.newton_schulz(G)
        ws = torch.full((max(256, gg.newton_schulz_workspace_size(2, M, N)),), 255, dtype=torch.uint8, device="cuda")
        again = gg.newton_schulz(G, workspace=ws)              # a workspace full of NaN patterns
        assert torch.equal(want, again)
        assert gg.newton_schulz(G, out=G) is G
        assert torch.equal(G, want)
    say("newton_schulz empty batch")
    assert gg.newton_schulz(torch.empty(0, 64, 64, device="cuda")).shape == (0, 64, 64)


def test_streams():
    """Two calls at once on two streams, each with its own workspace."""
    G = [gradient(4, 256, 320, k).cuda() for k in range(2)]
    want = [gg.newton_schulz(g) for g in G]
    torch.cuda.synchronize()
    say("newton_schulz on two streams")
    S = [torch.cuda.Stream() for _ in G]
    for _ in range(3):
        got = [gg.newton_schulz(g, stream=s) for g, s in zip(G, S)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,N", [(30, 200), (200, 300), (60, 200)])
def test_captured_and_replayed(M, N):
    W = torch.randn(2, M, N, device="cuda")
    mom, dW, Wc = torch.zeros_like(W), torch.zeros_like(W), torch.empty_like(W, dtype=torch.bfloat16)
    W2, mom2 = W.clone(), mom.clone()
    gg.newton_schulz(W)
    torch.cuda.synchronize()
    say(f"muon_step captured {M}x{N}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gg.muon_step(W, dW, mom, 0.02, W_bf16=Wc)
    for k in range(4):
        dW.copy_(gradient(2, M, N, k))
        graph.replay()
        torch.cuda.synchronize()
        gg.muon_step(W2, dW, mom2, 0.02)
        torch.cuda.synchronize()
        assert torch.equal(W, W2) and torch.equal(mom, mom2) and torch.equal(Wc, W2.bfloat16()), k


@pytest.mark.parametrize("coeffs,steps", [(MUON, 6), ((1.5, -0.5, 0.0), 7), ((12.0, -30.0, 20.0), 2), ((4.0, -6.0, 3.0), 3)])
def test_muon_step_batches_with_coefficients(coeffs, steps):
    """Coefficients whose steps taken together would lose what each keeps are taken one by one."""
    B, M, N = 16, 256, 512
    g = torch.Generator(device="cuda").manual_seed(steps)
    dW = 1e-3 * torch.randn(B, M, N, generator=g, device="cuda")
    dW[:, :16] *= 8
    W, mom = torch.zeros_like(dW), torch.zeros_like(dW)
    say(f"muon_step {B}x{M}x{N} {coeffs} steps{steps}")
    gg.muon_step(W, dW, mom, -1.0, beta=0.0, scale=1.0, steps=steps, coeffs=coeffs)
    torch.cuda.synchronize()
    X = iterate(dW, steps, coeffs, 1e-7, torch.float64)
    norm = lambda t: t.square().sum((-1, -2)).sqrt()  # noqa: E731
    x32 = iterate(dW.cpu(), steps, coeffs, 1e-7, torch.float32).double().cuda()
    most = 8 * norm(x32 - X) + 16 * U * norm(X)
    assert (norm(W.double() - X) <= most).all(), f"{(norm(W.double() - X) / norm(X)).max()} of {(most / norm(X)).max()}"


def test_offsets_beyond_32_bits():
    """2.2e9 elements (8.7 GB a copy of X): the first matrix against 64 bits, the others, which are equal, against it."""
    B, M, N = 130, 1024, 16384
    g = torch.Generator(device="cuda").manual_seed(7)
    one = (1e-3 * torch.randn(1, M, N, generator=g, device="cuda")).bfloat16()
    G = one.expand(B, M, N).contiguous()
    say(f"newton_schulz {B}x{M}x{N} bf16")
    out = gg.newton_schulz(G)
    torch.cuda.synchronize()
    want = iterate(one, 5, MUON, 1e-7, torch.float64)
    norm = lambda t: t.double().square().sum().sqrt()  # noqa: E731
    assert norm(out[:1].double() - want) <= (2.0 ** -8 + 8 * 30 * U) * norm(want)
    assert all(torch.equal(out[k], out[0]) for k in range(1, B))
