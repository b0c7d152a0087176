"""Layer norm forward and backward on the GPU against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, D = row length):
 * h is exact: a fp32 sum rounded to the storage type, the oracle's own.
 * mean, var: a lane adds at most 16 NV <= 64 terms in order, then at most 20
   levels of a tree, so a sum of terms t is off by at most 84 u sum|t|; 1 / sqrt
   halves var's relative error and adds 3 u: rstd within 50 u.
 * y before its rounding: (h - mean) carries 85 u mean|h| + u |h|, times rstd |w|,
   and 54 u of itself from rstd and three products; then half a step of the type
   (the step at |y|) once.
 * dx: the two sums are each within 84 u of the sum of their terms' sizes,
   z within 4 u + (mean's part: exact here, mean is an input); bounded below by
   100 u rstd (|g| + mean|g| + |z| mean|g z|) (+ u |dx|), then half a step once.
 * dweight, dbias: a chain of at most T / 512 + 60 adds (a lane's rows, 3 shuffles, 16
   wavefronts, 32 partial rows of a slice, 16 slices), and 4 u for each product dy z.
"""
import numpy as np
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(T, D, dtype, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g) * (1 + 9 * (torch.rand(D, generator=g) < 0.02)) + 0.5 * torch.randn(D, generator=g)
    r = 0.3 * torch.randn(T, D, generator=g)
    w = 1 + 0.1 * torch.randn(D, generator=g)
    b = 0.1 * torch.randn(D, generator=g)
    dy = torch.randn(T, D, generator=g)
    dh = torch.randn(T, D, generator=g)
    return [t.to(TYPES[dtype]) for t in (x, r, w, b, dy, dh)]


def forward64(x, r, w, b, eps, rms):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h64 = h.double()
    mean = torch.zeros(h.shape[0], dtype=torch.float64) if rms else h64.mean(1)
    d = h64 - mean[:, None]
    rstd = 1 / torch.sqrt(d.square().mean(1) + eps)
    y = d * rstd[:, None]
    slack = 54 * U * y.abs() + (86 * U * h64.abs().mean(1, keepdim=True) + U * h64.abs()) * rstd[:, None]
    if w is not None:
        y, slack = y * w.double(), slack * w.double().abs()
    if b is not None:
        y = y + b.double()
        slack = slack + U * y.abs()
    return h, mean, rstd, y, slack


def backward64(h, dy, mean, rstd, w, dh):
    z = (h.double() - (0 if mean is None else mean.double()[:, None])) * rstd.double()[:, None]
    dy = dy.double()
    g = dy if w is None else dy * w.double()
    s = rstd.double()[:, None]
    dx = g - z * (g * z).mean(1, keepdim=True)
    size = g.abs() + z.abs() * (g * z).abs().mean(1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(1, keepdim=True)
        size = size + g.abs().mean(1, keepdim=True)
    dx, slack = dx * s, 100 * U * size * s
    if dh is not None:
        dx = dx + dh.double()
        slack = slack + U * dx.abs()
    return dx, slack, dy * z, dy


def within(got, want, slack, half, what):
    got = got.double().cpu()
    off = (got - want).abs() - slack - half * want.abs() * (1 + 2 ** -6)
    assert torch.isfinite(got).all(), what
    assert float(off.max()) <= 1e-37, f"{what}: over the bound by {float(off.max()):.3e}"


SHAPES = [(1, 1), (3, 2), (5, 7), (1, 768), (2, 768), (37, 768), (9, 64), (130, 257), (64, 1001), (33, 1024),
          (7, 1032), (19, 2047), (12, 2048), (6, 2056), (5, 4100), (4, 8192), (3, 8200), (2, 16384), (3, 16383),
          (5000, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_forward(T, D, dtype):
    import grouped_gemm_permute_amd as gg
    x, r, w, b, _, _ = inputs(T, D, dtype, 11 + T + D)
    for rms, res, affine in ((False, True, True), (True, False, True), (False, False, False), (True, True, True)):
        say(f"layer_norm T{T} D{D} {dtype} rms{rms} residual{res} affine{affine}")
        a = dict(residual=r.cuda() if res else None, rms=rms, eps=1e-5)
        ww, bb = (w, b) if affine else (None, None)
        o = gg.layer_norm(x.cuda(), None if ww is None else ww.cuda(), None if bb is None else bb.cuda(), **a)
        torch.cuda.synchronize()
        h, mean, rstd, y, slack = forward64(x, r if res else None, ww, bb, 1e-5, rms)
        assert torch.equal(o["h"].cpu(), h)
        assert (o["mean"] is None) == rms
        h64 = h.double()
        if not rms:
            within(o["mean"], mean, 86 * U * h64.abs().mean(1), 0, "mean")
        # a deviation is off by the mean's error and u of itself
        dev = 172 * U * h64.abs().mean(1) * ((h64 - mean[:, None]).abs().mean(1)) * rstd ** 3 if not rms else 0
        within(o["rstd"], rstd, 50 * U * rstd + dev, 0, "rstd")
        within(o["y"], y, slack, HALF[dtype], "y")


# the weight's gradients by partial rows (more than 1024 rows, or 512 with tails), and on both sides of that
TALL = [(1025, 1), (1026, 2), (1027, 7), (1025, 64), (1030, 257), (1026, 768), (1100, 1001), (1025, 1024), (1030, 1032),
        (1040, 2047), (1025, 2056), (1030, 4100), (1025, 8200), (1026, 16384), (513, 16383), (512, 1001), (513, 1001),
        (1024, 1000), (512, 12), (600, 20), (20000, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SHAPES + TALL)
def test_backward(T, D, dtype):
    import grouped_gemm_permute_amd as gg
    x, _, w, _, dy, dh = inputs(T, D, dtype, 5 + T + D)
    for rms, stream_grad, affine in ((False, True, True), (True, False, True), (False, False, False)):
        say(f"layer_norm_backward T{T} D{D} {dtype} rms{rms} dh{stream_grad} affine{affine}")
        _, mean, rstd, _, _ = forward64(x, None, None, None, 1e-5, rms)
        mean = None if rms else mean.float()
        rstd = rstd.float()
        ww = w if affine else None
        o = gg.layer_norm_backward(x.cuda(), dy.cuda(), rstd.cuda(), None if rms else mean.cuda(),
                                   None if ww is None else ww.cuda(), dh.cuda() if stream_grad else None,
                                   bias_grad=affine)
        torch.cuda.synchronize()
        dx, slack, tw, tb = backward64(x, dy, mean, rstd, ww, dh if stream_grad else None)
        within(o["dx"], dx, slack, HALF[dtype], "dx")
        if not affine:
            assert o["dweight"] is None and o["dbias"] is None
            continue
        adds = -(-T // 512) + 60
        within(o["dweight"], tw.sum(0), (adds + 4) * U * tw.abs().sum(0), 0, "dweight")
        within(o["dbias"], tb.sum(0), adds * U * tb.abs().sum(0), 0, "dbias")


def test_backward_against_differences():
    """dx, dweight, dbias against central differences of the forward formula in 64 bits."""
    import grouped_gemm_permute_amd as gg
    T, D, eps, d = 3, 37, 1e-5, 1e-6
    x, r, w, b, dy, _ = [t.double() for t in inputs(T, D, "f32", 3)]
    for rms in (False, True):
        def loss(x, w, b):
            m = 0 if rms else x.mean(1, keepdim=True)
            v = (x - m).square().mean(1, keepdim=True)
            return (((x - m) / torch.sqrt(v + eps) * w + b) * dy).sum()

        say(f"layer_norm differences rms{rms}")
        f = gg.layer_norm(x.float().cuda(), w.float().cuda(), b.float().cuda(), rms=rms)
        o = gg.layer_norm_backward(f["h"], dy.float().cuda(), f["rstd"], f["mean"], w.float().cuda(), bias_grad=True)
        torch.cuda.synchronize()
        x, w, b = x.float().double(), w.float().double(), b.float().double()
        for name, t, at in (("dx", x, 0), ("dweight", w, 1), ("dbias", b, 2)):
            num = torch.zeros_like(t)
            for i in np.ndindex(*t.shape):
                args = [x, w, b]
                hi, lo = t.clone(), t.clone()
                hi[i] += d
                lo[i] -= d
                args[at] = hi
                up = loss(*args)
                args[at] = lo
                num[i] = (up - loss(*args)) / (2 * d)
            # differences: d^2 (third derivatives, of order 1) and 2^-52 |loss| / d ~ 1e-8; the kernel 1e-5 of the largest
            assert float((o[name].double().cpu() - num).abs().max()) < 1e-5 * float(num.abs().max()) + 1e-7, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_do_not_touch_each_other(dtype):
    """A row with an infinity or a NaN is NaN by itself; constant and zero rows are finite; a large row does not overflow its mean."""
    import grouped_gemm_permute_amd as gg
    D = 300
    x = torch.randn(6, D).to(TYPES[dtype])
    x[1, 7] = float("inf")
    x[2, 299] = float("nan")
    x[3] = 0
    x[4] = 5
    say(f"layer_norm special rows {dtype}")
    o = gg.layer_norm(x.cuda())
    y = o["y"].cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert (y[3] == 0).all() and (y[4] == 0).all()
    assert torch.isfinite(y[[0, 5]]).all()
    alone = gg.layer_norm(x[[0, 5]].contiguous().cuda())["y"].cpu()
    assert torch.equal(alone, y[[0, 5]])


def test_empty_in_place_and_stream():
    import grouped_gemm_permute_amd as gg
    say("layer_norm T0")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert gg.layer_norm(e, w, w)["y"].shape == (0, 64)
    o = gg.layer_norm_backward(e, e, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), w, bias_grad=True,
                               out={"dweight": torch.full((64,), 3.0, device="cuda")})
    assert (o["dweight"] == 0).all() and (o["dbias"] == 0).all()

    x, r, w, b, dy, dh = [t.cuda() for t in inputs(700, 100, "bf16", 9)]
    want = gg.layer_norm(x, w, b, residual=r)
    back = gg.layer_norm_backward(want["h"], dy, want["rstd"], want["mean"], w, dh, bias_grad=True)
    say("layer_norm in place")
    x2, r2 = x.clone(), r.clone()
    got = gg.layer_norm(x2, w, b, residual=r2, out={"y": x2, "h": r2})
    assert torch.equal(x2, want["y"]) and torch.equal(r2, want["h"]) and torch.equal(got["rstd"], want["rstd"])
    dh2 = dh.clone()
    got = gg.layer_norm_backward(want["h"], dy, want["rstd"], want["mean"], w, dh2, bias_grad=True, out={"dx": dh2})
    assert torch.equal(dh2, back["dx"]) and torch.equal(got["dweight"], back["dweight"])
    say("layer_norm on another stream")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gg.layer_norm(x, w, b, residual=r, stream=s)
    gb = gg.layer_norm_backward(got["h"], dy, got["rstd"], got["mean"], w, dh, bias_grad=True, stream=s)
    s.synchronize()
    assert torch.equal(got["y"], want["y"])
    assert all(torch.equal(gb[k], back[k]) for k in ("dx", "dweight", "dbias"))


def test_captured_and_replayed():
    import grouped_gemm_permute_amd as gg
    x, r, w, b, dy, dh = [t.cuda() for t in inputs(1000, 768, "bf16", 21)]

    def step():
        f = gg.layer_norm(x, w, b, residual=r)
        g = gg.layer_norm_backward(f["h"], dy, f["rstd"], f["mean"], w, dh, bias_grad=True)
        return f["y"], g["dx"], g["dweight"], g["dbias"]

    step()
    torch.cuda.synchronize()
    say("layer_norm captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(inputs(1000, 768, "bf16", 30 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


@pytest.mark.parametrize("T", [37, 1025])
@pytest.mark.parametrize("D,dtype", [(5, "bf16"), (777, "f32"), (5001, "bf16"), (8193, "bf16"), (16383, "f32"), (16384, "bf16")])
def test_in_place_rows_of_every_width(T, D, dtype):
    """y over x, h over the residual, dx over dy, dh or h: rows of one lane's group to a whole workgroup, with tails."""
    import grouped_gemm_permute_amd as gg
    x, r, w, b, dy, dh = [t.cuda() for t in inputs(T, D, dtype, 4)]
    for rms in (False, True):
        say(f"layer_norm in place T{T} D{D} {dtype} rms{rms}")
        want = gg.layer_norm(x, w, b, residual=r, rms=rms)
        x2, r2 = x.clone(), r.clone()
        gg.layer_norm(x2, w, b, residual=r2, rms=rms, out={"y": x2, "h": r2})
        assert torch.equal(x2, want["y"]) and torch.equal(r2, want["h"])
        x2, r2 = x.clone(), r.clone()
        gg.layer_norm(x2, w, b, residual=r2, rms=rms, out={"y": r2, "h": x2})
        assert torch.equal(r2, want["y"]) and torch.equal(x2, want["h"])
        back = gg.layer_norm_backward(want["h"], dy, want["rstd"], want["mean"], w, dh, bias_grad=True)
        for which in range(3):
            t = [want["h"].clone(), dy.clone(), dh.clone()]
            got = gg.layer_norm_backward(t[0], t[1], want["rstd"], want["mean"], w, t[2], bias_grad=True,
                                         out={"dx": t[which]})
            assert all(torch.equal(got[k], back[k]) for k in ("dx", "dweight", "dbias")), which


def test_offsets_beyond_32_bits():
    """2.4e9 elements: the last rows as by themselves, and the weight's gradient as many times that of one part."""
    import grouped_gemm_permute_amd as gg
    T, D, part = 600000, 4096, 600
    x, _, w, b, dy, _ = [t.cuda() for t in inputs(part, D, "bf16", 3)]
    X, DY = x.repeat(T // part, 1), dy.repeat(T // part, 1)
    say(f"layer_norm {T}x{D} bf16")
    f = gg.layer_norm(X, w, b)
    g = gg.layer_norm_backward(X, DY, f["rstd"], f["mean"], w, bias_grad=True)
    torch.cuda.synchronize()
    f1 = gg.layer_norm(x, w, b)
    g1 = gg.layer_norm_backward(x, dy, f1["rstd"], f1["mean"], w, bias_grad=True)
    for got, want in ((f["y"], f1["y"]), (g["dx"], g1["dx"])):
        assert all(torch.equal(got[k:k + part], want) for k in range(0, T, part * 37)) and torch.equal(got[-part:], want)
    z = (x.double() - f1["mean"].double()[:, None]) * f1["rstd"].double()[:, None]
    for got, terms in ((g["dweight"], dy.double() * z), (g["dbias"], dy.double())):
        # sums of at most T / 512 terms in a row, then 512 partial rows: u (T / 512 + 16 + 16) of the terms' sum
        most = 2.0 ** -24 * (T / 512 + 32 + 4) * terms.abs().sum(0) * (T // part)
        assert ((got.double() - terms.sum(0) * (T // part)).abs() <= most).all()
