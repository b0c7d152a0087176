"""Layer norm at its edges: in place without a residual."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 768), (3, 7), (40, 1001), (5, 5000), (2, 16384)])
def test_in_place_without_a_residual(T, D, dtype):
    """y over x: the row the backward needs is gone, so no h is handed out (x would be y)."""
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(D)).to(TYPES[dtype]).cuda()
    w = torch.randn(D, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype]).cuda()
    for rms in (False, True):
        say(f"layer_norm in place T{T} D{D} {dtype} rms{rms}")
        want = gg.layer_norm(x, w, rms=rms)
        assert want["h"] is x
        x2 = x.clone()
        got = gg.layer_norm(x2, w, rms=rms, out={"y": x2})
        assert got["y"] is x2 and torch.equal(x2, want["y"]) and torch.equal(got["rstd"], want["rstd"])
        assert got["h"] is None
        y = torch.empty_like(x)
        assert gg.layer_norm(x, w, rms=rms, out={"y": y})["h"] is x
        # with a residual the sum has its own place, and y may still be x
        r = torch.ones_like(x)
        sums = gg.layer_norm(x, w, residual=r, rms=rms)
        x2, h = x.clone(), torch.empty_like(x)
        got = gg.layer_norm(x2, w, residual=r, rms=rms, out={"y": x2, "h": h})
        assert got["h"] is h and torch.equal(h, sums["h"]) and torch.equal(x2, sums["y"])
    empty = torch.empty(0, D, dtype=TYPES[dtype], device="cuda")
    assert gg.layer_norm(empty)["h"] is empty
