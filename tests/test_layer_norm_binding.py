"""Layer norm: what the C entry points and the binding refuse on the host
(no GPU needed; no pointer here is dereferenced)."""
import pytest
import torch

gg = pytest.importorskip("grouped_gemm_permute_amd")
from grouped_gemm_permute_amd import _lib as L  # noqa: E402

FAKE = 0x7F0000000000


def _fwd(**over):
    a = dict(x=FAKE, r=None, w=FAKE, b=FAKE, y=FAKE, h=None, mean=FAKE, rstd=FAKE, T=16, D=64, rms=0,
             eps=1e-5, dt=L.MOE_BF16)
    a.update(over)
    return L.lib().moe_layer_norm_forward(a["x"], a["r"], a["w"], a["b"], a["y"], a["h"], a["mean"],
                                          a["rstd"], a["T"], a["D"], a["rms"], a["eps"], a["dt"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), L.MOE_ERR_INVALID_ARG),
    (dict(y=None), L.MOE_ERR_INVALID_ARG),
    (dict(x=FAKE + 8), L.MOE_ERR_INVALID_ARG),
    (dict(w=FAKE + 2), L.MOE_ERR_INVALID_ARG),
    (dict(mean=FAKE + 2), L.MOE_ERR_INVALID_ARG),
    (dict(r=FAKE), L.MOE_ERR_INVALID_ARG),               # a residual without a place for the sum
    (dict(h=FAKE), L.MOE_ERR_INVALID_ARG),
    (dict(rms=1), L.MOE_ERR_INVALID_ARG),                # rms has no mean
    (dict(eps=-1.0), L.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), L.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), L.MOE_ERR_INVALID_ARG),
    (dict(T=-1), L.MOE_ERR_INVALID_ARG),
    (dict(T=1 << 31), L.MOE_ERR_INVALID_ARG),
    (dict(D=0), L.MOE_ERR_INVALID_ARG),
    (dict(dt=4), L.MOE_ERR_INVALID_ARG),
    (dict(D=16385), L.MOE_ERR_UNSUPPORTED),
    (dict(T=0, x=None, y=None), L.MOE_OK),
])
def test_forward_refusals(over, status):
    assert _fwd(**over) == status


def _bwd(**over):
    a = dict(h=FAKE, mean=FAKE, rstd=FAKE, w=FAKE, dy=FAKE, dh=None, dx=FAKE, dw=FAKE, db=FAKE, T=2000, D=64,
             dt=L.MOE_BF16, ws=FAKE, n=1 << 30)
    a.update(over)
    return L.lib().moe_layer_norm_backward(a["h"], a["mean"], a["rstd"], a["w"], a["dy"], a["dh"], a["dx"],
                                           a["dw"], a["db"], a["T"], a["D"], a["dt"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(h=None), L.MOE_ERR_INVALID_ARG),
    (dict(rstd=None), L.MOE_ERR_INVALID_ARG),
    (dict(dx=None), L.MOE_ERR_INVALID_ARG),
    (dict(dh=FAKE + 4), L.MOE_ERR_INVALID_ARG),
    (dict(dw=FAKE + 2), L.MOE_ERR_INVALID_ARG),
    (dict(ws=None), L.MOE_ERR_INVALID_ARG),
    (dict(ws=FAKE + 64), L.MOE_ERR_INVALID_ARG),
    (dict(n=255), L.MOE_ERR_WORKSPACE),
    (dict(T=-1), L.MOE_ERR_INVALID_ARG),
    (dict(D=20000), L.MOE_ERR_UNSUPPORTED),
    (dict(dt=9), L.MOE_ERR_INVALID_ARG),
    (dict(T=0, dw=None, db=None), L.MOE_OK),
])
def test_backward_refusals(over, status):
    assert _bwd(**over) == status


def test_workspace_size():
    size = L.lib().moe_layer_norm_backward_workspace_size
    assert size(0, 64, L.MOE_BF16) == 0
    assert size(1025, 64, L.MOE_BF16) == 33 * 2 * 64 * 4             # partial rows of each sum, one of 32 rows
    assert size(1, 64, L.MOE_BF16) == size(512, 1001, L.MOE_F32) == size(1024, 1000, L.MOE_F32) == 0   # few rows
    assert size(513, 1001, L.MOE_F32) > 0
    assert size(1 << 20, 768, L.MOE_BF16) <= 512 * 2 * 768 * 4
    assert size(4, 20000, L.MOE_BF16) == 0 and size(-1, 64, L.MOE_BF16) == 0


def test_binding_refusals():
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        gg.layer_norm(x, w, w)
    with pytest.raises(TypeError, match="weight"):
        gg.layer_norm(x, w.float(), w)
    with pytest.raises(ValueError, match="bias"):
        gg.layer_norm(x, w, w[:32])
    with pytest.raises(ValueError, match="residual"):
        gg.layer_norm(x, residual=x[:4])
    with pytest.raises(ValueError, match="contiguous"):
        gg.layer_norm(torch.zeros(64, 8, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="T,D"):
        gg.layer_norm(x[0])
    with pytest.raises(TypeError, match="dtype"):
        gg.layer_norm(x.half())
    with pytest.raises(ValueError, match="place for h"):
        gg.layer_norm(x, out={"h": x})
    s = torch.zeros(8)
    with pytest.raises(TypeError, match="dy"):
        gg.layer_norm_backward(x, x.float(), s, s, w)
    with pytest.raises(ValueError, match="rstd"):
        gg.layer_norm_backward(x, x, s[:4], s, w)
    with pytest.raises(TypeError, match="mean"):
        gg.layer_norm_backward(x, x, s, s.double(), w)
    with pytest.raises(ValueError, match="place for dweight"):
        gg.layer_norm_backward(x, x, s, s, out={"dweight": s})
    with pytest.raises(ValueError, match="GPU"):
        gg.layer_norm_backward(x, x, s, s, w)
