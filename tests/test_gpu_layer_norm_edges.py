"""Layer norm at its edges: in place without a residual, rows whose mean times rstd passes fp32's range, infinite and NaN
rows of the root mean square norm."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 1030])
@pytest.mark.parametrize("D", [1, 2, 4, 8, 37, 100, 777, 1001, 2056, 5000, 9000, 12289])
def test_backward_where_mean_times_rstd_overflows(T, D, dtype):
    """Rows of one value, 2^121, with rstd 2^8: every z is 0 although mean rstd is beyond fp32, so
    dx = rstd (g - sum(g) / D).  g are small whole numbers and D of them sum exactly, so dx is off by the rounding of
    1 / D, of its product and of the difference, times rstd (u = 2^-24 of |g| + |mean|), and half a step of the type."""
    dt = TYPES[dtype]
    h = torch.full((T, D), 2.0**121, dtype=dt, device="cuda")
    mean, rstd = torch.full((T,), 2.0**121, device="cuda"), torch.full((T,), 2.0**8, device="cuda")
    dy = torch.randint(-3, 4, (T, D), generator=torch.Generator().manual_seed(D)).to(dt).cuda()
    say(f"layer_norm_backward mean rstd over fp32 T{T} D{D} {dtype}")
    o = gg.layer_norm_backward(h, dy, rstd, mean, torch.ones(D, dtype=dt, device="cuda"), bias_grad=True)
    torch.cuda.synchronize()
    g = dy.double()
    m = g.mean(1, keepdim=True)
    want = 2.0**8 * (g - m)
    most = 4 * 2.0**-24 * 2.0**8 * (g.abs() + m.abs()) + (2.0**-8 if dtype == "bf16" else 2.0**-24) * want.abs() * 1.01
    assert ((o["dx"].double() - want).abs() <= most).all()
    assert (o["dweight"] == 0).all() and torch.equal(o["dbias"].double(), g.sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [5, 300, 1032, 5000, 9000])
def test_rms_rows_with_infinities_and_nan(D, dtype):
    """Beside an infinity a root mean square row is 0 (1 / sqrt(inf)), the infinity itself NaN; a NaN takes its whole row;
    the other rows are untouched, and so is the largest row whose squares fp32 still holds."""
    x = torch.randn(6, D, generator=torch.Generator().manual_seed(D)).to(TYPES[dtype])
    x[1, D // 2] = float("inf")
    x[2, D - 1] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = 1e17      # D squares of 1e34 sum to at most 1e38
    say(f"layer_norm rms special rows D{D} {dtype}")
    y = gg.layer_norm(x.cuda(), rms=True)["y"].float().cpu()
    for row, at in ((1, D // 2), (3, 0)):
        assert torch.isnan(y[row, at])
        assert (torch.cat([y[row, :at], y[row, at + 1:]]) == 0).all()
    assert torch.isnan(y[2]).all()
    assert ((y[4] - 1).abs() <= 2.0**-8).all()
    alone = gg.layer_norm(x[[0, 5]].contiguous().cuda(), rms=True)["y"].float().cpu()
    assert torch.equal(alone, y[[0, 5]])
