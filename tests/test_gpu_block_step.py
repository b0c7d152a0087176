"""A training step around the layer, its operators one after the other as a
program calls them: residual sum and norm, router, layer (its gate and up
products kept), the layer's backward, the norm's backward with the residual
stream's gradient, and a Muon step on every expert matrix from the gradients
that the backward wrote.

In fp32 the whole chain is compared with torch autograd in 64 bits: each stage
is within 1e-5 of its largest output (the layer's own bound; the norms' are
smaller), no stage after the first multiplies an error by more than about 2
relative to its output, so 5e-5 of the largest bounds the end.  In bf16 each
stage is compared with its formula in 64 bits on the inputs it was given.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_permute_amd as gg
import oracle
from gpu_util import check_close, oracle_threads, say, to_f64
from test_gpu_layer_norm import HALF, backward64, forward64, within
from test_gpu_muon import MUON, U, iterate

pytestmark = pytest.mark.gpu
LR, BETA, DECAY = 0.02, 0.95, 0.1


def block(T, D, F, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, by=1.0):
        return (torch.randn(shape, generator=g) * by).to(dtype).cuda()

    p = dict(x=n(T, D), r=n(T, D, by=0.5), ln_w=n(D, by=0.1) + 1, ln_b=n(D, by=0.1), gate=n(D, E, by=D ** -0.5),
             W1=n(E, D, F, by=D ** -0.5), W3=n(E, D, F, by=D ** -0.5), W2=n(E, F, D, by=F ** -0.5),
             Ws1=n(D, F, by=D ** -0.5), Ws3=n(D, F, by=D ** -0.5), Ws2=n(F, D, by=F ** -0.5), dout=n(T, D))
    for name in ("W1", "W3", "W2"):
        p["master_" + name] = p[name].float()
        p["mom_" + name] = torch.zeros(p[name].shape, device="cuda")
    return p


def step(p, k=2):
    """One step; weights and momenta are updated in place."""
    shared = (p["Ws1"], p["Ws3"], p["Ws2"])
    f = gg.layer_norm(p["x"], p["ln_w"], p["ln_b"], residual=p["r"])
    idx, w = gg.router_topk(f["y"], p["gate"], k)
    layer = (f["y"], idx, w, p["W1"], p["W3"], p["W2"], shared)
    if p["x"].dtype == torch.bfloat16:
        y, gu = gg.forward_save_gu(*layer)
    else:
        y, gu = gg.forward(*layer), None
    out = y + f["h"]
    g = gg.backward(*layer, p["dout"], gu=gu)
    b = gg.layer_norm_backward(f["h"], g["dx"], f["rstd"], f["mean"], p["ln_w"], dh=p["dout"], bias_grad=True)
    for name in ("W1", "W3", "W2"):
        bf16 = p["x"].dtype == torch.bfloat16
        gg.muon_step(p["master_" + name], g["d" + name], p["mom_" + name], LR, beta=BETA, weight_decay=DECAY,
                     W_bf16=p[name] if bf16 else None)
    return dict(f=f, idx=idx, w=w, y=y, out=out, g=g, b=b)


def muon64(W0, dW, half):
    """(new W, bound) of a first step from zero momentum."""
    f = lambda v: torch.tensor(v, dtype=torch.float32).double().item()  # noqa: E731
    u = dW.double() + f(BETA) * dW.double()
    X, X32 = iterate(u, 5, MUON, 1e-7, torch.float64), iterate(u.float(), 5, MUON, 1e-7, torch.float32).double()
    rate = f(LR) * max(1.0, W0.shape[2] / W0.shape[1]) ** 0.5
    want = (1 - f(LR) * f(DECAY)) * W0.double() - rate * X
    off = 8 * (X32 - X).square().sum((-1, -2), keepdim=True).sqrt() + 16 * U * X.abs().amax((-1, -2), keepdim=True)
    return want, rate * off + 4 * U * (W0.double().abs() + rate * X.abs()) + half * want.abs() * 1.01


def test_fp32_step_against_autograd():
    T, D, F, E = 150, 64, 96, 4
    say(f"block step fp32 T{T} D{D} F{F} E{E}")
    p = block(T, D, F, E, torch.float32, 3)
    W0 = {n: p[n].cpu() for n in ("W1", "W3", "W2")}
    r = step(p)
    torch.cuda.synchronize()
    leaf = {n: p[n].cpu().double().requires_grad_() for n in ("x", "ln_w", "ln_b", "Ws1", "Ws3", "Ws2")}
    leaf.update({n: W0[n].double().requires_grad_() for n in W0})
    h = leaf["x"] + p["r"].cpu().double()
    d = h - h.mean(1, keepdim=True)
    y = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * leaf["ln_w"] + leaf["ln_b"]
    ffn = lambda v, a, c, b: (torch.nn.functional.silu(v @ a) * (v @ c)) @ b  # noqa: E731
    out = h + ffn(y, leaf["Ws1"], leaf["Ws3"], leaf["Ws2"])
    idx, w = r["idx"].cpu().long(), r["w"].cpu().double()      # the routing is given: no gradient through it
    each = torch.stack([ffn(y, leaf["W1"][e], leaf["W3"][e], leaf["W2"][e]) for e in range(E)], 1)
    out = out + (each.gather(1, idx[:, :, None].expand(-1, -1, D)) * w[:, :, None]).sum(1)
    (out * p["dout"].cpu().double()).sum().backward()
    got = {"out": (r["out"], out.detach()), "dx": (r["b"]["dx"], leaf["x"].grad),
           "ln_w": (r["b"]["dweight"], leaf["ln_w"].grad), "ln_b": (r["b"]["dbias"], leaf["ln_b"].grad)}
    got.update({n: (r["g"]["d" + n], leaf[n].grad) for n in ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2")})
    for name, (a, want) in got.items():
        off = float((a.double().cpu() - want).abs().max())
        assert off <= 5e-5 * float(want.abs().max()), f"{name}: {off:.2e} of {float(want.abs().max()):.2e}"
    for n in ("W1", "W3", "W2"):
        want, most = muon64(W0[n], r["g"]["d" + n].cpu(), U)
        assert ((p["master_" + n].double().cpu() - want).abs() <= most).all(), n


def test_bf16_step_by_stages():
    T, D, F, E = 700, 128, 256, 8
    say(f"block step bf16 T{T} D{D} F{F} E{E}")
    p = block(T, D, F, E, torch.bfloat16, 5)
    before = {n: p[n].clone() for n in ("W1", "W3", "W2")}
    r = step(p)
    torch.cuda.synchronize()
    cpu = lambda t: t.cpu()  # noqa: E731
    h, mean, rstd, y, slack = forward64(cpu(p["x"]), cpu(p["r"]), cpu(p["ln_w"]), cpu(p["ln_b"]), 1e-5, False)
    assert torch.equal(r["f"]["h"].cpu(), h)
    within(r["f"]["y"], y, slack, HALF["bf16"], "norm")
    n64 = lambda t: np.ascontiguousarray(to_f64(t))  # noqa: E731
    layer = [n64(r["f"]["y"]), r["idx"].cpu().numpy(), r["w"].cpu().numpy(),
             *[n64(before[n]) for n in ("W1", "W3", "W2")], tuple(n64(p[n]) for n in ("Ws1", "Ws3", "Ws2"))]
    check_close(to_f64(r["y"]), oracle.forward_dense(*layer, nthreads=oracle_threads()), "bf16", "layer")
    ref = oracle.backward(*layer, n64(p["dout"]), nthreads=oracle_threads())
    for n in ("dx", "dW1", "dW3", "dW2"):
        check_close(to_f64(r["g"][n]), ref[n], "bf16", n)
    dx, slack, tw, tb = backward64(h, cpu(r["g"]["dx"]), cpu(r["f"]["mean"]), cpu(r["f"]["rstd"]), cpu(p["ln_w"]),
                                   cpu(p["dout"]))
    within(r["b"]["dx"], dx, slack, HALF["bf16"], "norm dx")
    within(r["b"]["dweight"], tw.sum(0), 70 * U * tw.abs().sum(0), 0, "norm dweight")
    within(r["b"]["dbias"], tb.sum(0), 70 * U * tb.abs().sum(0), 0, "norm dbias")
    for n in ("W1", "W3", "W2"):
        want, most = muon64(before[n].float().cpu(), r["g"]["d" + n].cpu(), U)
        assert ((p["master_" + n].double().cpu() - want).abs() <= most).all(), n
        assert torch.equal(p[n], p["master_" + n].bfloat16())


def test_captured_step_is_the_eager_step():
    """The step captured once and replayed four times, beside the same steps run eagerly."""
    T, D, F, E = 600, 128, 256, 8
    a, b = block(T, D, F, E, torch.bfloat16, 9), block(T, D, F, E, torch.bfloat16, 9)
    step(block(T, D, F, E, torch.bfloat16, 9))
    torch.cuda.synchronize()
    say("block step captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(a)
    for k in range(4):
        x = block(T, D, F, E, torch.bfloat16, 20 + k)["x"]
        a["x"].copy_(x)
        b["x"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        e = step(b)
        torch.cuda.synchronize()
        assert torch.equal(r["out"], e["out"]) and torch.equal(r["b"]["dx"], e["b"]["dx"])
        assert torch.equal(r["b"]["dweight"], e["b"]["dweight"])
        for n in ("W1", "W3", "W2"):
            assert torch.equal(a[n], b[n]) and torch.equal(a["mom_" + n], b["mom_" + n]), (k, n)
