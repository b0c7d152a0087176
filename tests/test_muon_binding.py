"""Newton-Schulz and Muon step: what the C entry points and the binding
refuse on the host (no GPU needed; no pointer here is dereferenced)."""
import pytest
import torch

gg = pytest.importorskip("grouped_gemm_permute_amd")
from grouped_gemm_permute_amd import _lib as L  # noqa: E402

FAKE = 0x7F0000000000
NAN, INF = float("nan"), float("inf")
BAD, UNS = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED

COMMON = [
    (dict(B=-1), BAD), (dict(M=0), BAD), (dict(N=-3), BAD),
    (dict(steps=0), BAD), (dict(steps=65), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD),
    (dict(a=NAN), BAD), (dict(c=INF), BAD),
    (dict(dt=5), BAD), (dict(ws=None), BAD), (dict(ws=FAKE + 128), BAD),
    (dict(n=1024), L.MOE_ERR_WORKSPACE),
    (dict(M=32769), UNS), (dict(B=65536), UNS),
    (dict(B=65535, M=4096, N=4096), UNS),                       # 2^24 tiles and more
    (dict(a=20.0), UNS), (dict(c=-500.0), UNS),                 # singular values would run away
    (dict(a=0.1, b=0.0, c=0.0, steps=12), UNS), (dict(a=0.0, b=1e-13, c=0.0), UNS),     # or vanish
    (dict(a=0.1, b=0.0, c=0.0, steps=9, B=0), L.MOE_OK), (dict(a=0.0, b=0.0, c=0.0, B=0), L.MOE_OK),
    (dict(B=0), L.MOE_OK),
]


def _ns(**over):
    x = dict(G=FAKE, out=FAKE, B=2, M=64, N=100, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, dt=L.MOE_F32,
             ws=FAKE, n=1 << 62)
    x.update(over)
    return L.lib().moe_newton_schulz(x["G"], x["out"], x["B"], x["M"], x["N"], x["steps"], x["a"], x["b"], x["c"],
                                     x["eps"], x["dt"], x["ws"], x["n"], None)


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(G=None), BAD), (dict(out=None), BAD), (dict(G=FAKE + 4), BAD), (dict(out=FAKE + 8), BAD)])
def test_newton_schulz_refusals(over, status):
    assert _ns(**over) == status


def _muon(**over):
    x = dict(W=FAKE, Wc=None, dW=FAKE, m=FAKE, B=2, M=64, N=100, lr=0.02, beta=0.95, wd=0.0, scale=1.0, nest=1,
             steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, dt=L.MOE_F32, ws=FAKE, n=1 << 62)
    x.update(over)
    return L.lib().moe_muon_step(x["W"], x["Wc"], x["dW"], x["m"], x["B"], x["M"], x["N"], x["lr"], x["beta"],
                                 x["wd"], x["scale"], x["nest"], x["steps"], x["a"], x["b"], x["c"], x["eps"],
                                 x["dt"], x["ws"], x["n"], None)


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(W=None), BAD), (dict(dW=None), BAD), (dict(m=None), BAD), (dict(m=FAKE + 4), BAD),
    (dict(Wc=FAKE + 2), BAD), (dict(Wc=FAKE, dt=L.MOE_BF16), BAD),
    (dict(lr=NAN), BAD), (dict(beta=INF), BAD), (dict(wd=NAN), BAD), (dict(scale=INF), BAD)])
def test_muon_refusals(over, status):
    assert _muon(**over) == status


def test_workspace_size():
    size = gg.newton_schulz_workspace_size
    assert size(4, 32, 256) == 0 and size(4, 384, 8) == 0            # one workgroup a matrix, no workspace
    assert size(4, 5000, 8) == 4 * 40 * 2048 and size(2, 32, 257) == 2 * 3 * 3 * 2048    # chunks' sums of A
    assert size(1, 33, 33) > 0 and size(1, 0, 5) == 0 and size(0, 64, 64) == 0
    assert size(8, 768, 1536) == size(8, 1536, 768)
    assert size(8, 768, 1536) < 8 * (12 * 768 * 1536 + 20 * 768 * 768) + (1 << 16)


def test_binding_refusals():
    G = torch.zeros(2, 64, 48)
    with pytest.raises(ValueError, match="GPU"):
        gg.newton_schulz(G)
    with pytest.raises(TypeError, match="dtype"):
        gg.newton_schulz(G.half())
    with pytest.raises(ValueError, match="M,N"):
        gg.newton_schulz(G[None])
    with pytest.raises(ValueError, match="contiguous"):
        gg.newton_schulz(G.transpose(1, 2))
    with pytest.raises(TypeError, match="out"):
        gg.newton_schulz(G, out=G.bfloat16())
    W = G.bfloat16()
    with pytest.raises(TypeError, match="dW"):
        gg.muon_step(W, W, G, 0.1)
    with pytest.raises(ValueError, match="momentum"):
        gg.muon_step(W, G, G[:1], 0.1)
    with pytest.raises(ValueError, match="fp32 W"):
        gg.muon_step(W, G, G, 0.1, W_bf16=W)
    with pytest.raises(TypeError, match="W_bf16"):
        gg.muon_step(G, G, G, 0.1, W_bf16=G)
    with pytest.raises(ValueError, match="GPU"):
        gg.muon_step(W, G, G, 0.1)
