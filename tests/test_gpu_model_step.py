"""A one-block model's training step with a vocabulary at both ends, its operators one after the other as a program calls
them: tokens looked up, residual sum and norm, router, layer, last norm, cross entropy over the same table, and back, the
table's gradient from both ends.

In fp32 the whole chain is compared with torch autograd in 64 bits, with the bound of the block's own test: each stage is within
1e-5 of its largest output, none after the first multiplies an error by more than about 2 relative to its output, and these are
three stages more: 1e-4 of the largest bounds the end.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say

pytestmark = pytest.mark.gpu


def model(T, D, F, E, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, by=1.0):
        return (torch.randn(shape, generator=g) * by).to(dtype).cuda()

    p = dict(table=n(V, D, by=D ** -0.5), ln_w=n(D, by=0.1) + 1, ln_b=n(D, by=0.1), out_w=n(D, by=0.1) + 1, out_b=n(D, by=0.1),
             gate=n(D, E, by=D ** -0.5), W1=n(E, D, F, by=D ** -0.5), W3=n(E, D, F, by=D ** -0.5), W2=n(E, F, D, by=F ** -0.5))
    p["ids"] = torch.randint(0, V, (T,), generator=g).int().cuda()
    p["targets"] = torch.randint(-2, V, (T,), generator=g).int().cuda()     # a few without one
    p["dtable"] = torch.zeros(V, D, device="cuda")
    return p


def step(p, k=2):
    V, D = p["table"].shape
    scale = D ** 0.5
    x = gg.embedding(p["ids"], p["table"], scale=scale)
    f = gg.layer_norm(x, p["ln_w"], p["ln_b"])
    idx, w = gg.router_topk(f["y"], p["gate"], k)
    layer = (f["y"], idx, w, p["W1"], p["W3"], p["W2"], None)
    y = gg.forward(*layer)
    last = gg.layer_norm(y, p["out_w"], p["out_b"], residual=x)
    ce = gg.cross_entropy(last["y"], p["table"], p["targets"])
    mean = torch.full_like(ce["loss"], 1.0 / len(ce["loss"]))
    b = gg.cross_entropy_backward(last["y"], p["table"], p["targets"], ce["lse"], mean, out={"dW": p["dtable"]})
    lb = gg.layer_norm_backward(last["h"], b["dh"], last["rstd"], last["mean"], p["out_w"], bias_grad=True)
    g = gg.backward(*layer, lb["dx"])
    nb = gg.layer_norm_backward(f["h"], g["dx"], f["rstd"], f["mean"], p["ln_w"], dh=lb["dx"], bias_grad=True)
    gg.embedding_backward(p["ids"], nb["dx"], V, scale=scale, out=p["dtable"], accumulate=True)
    return dict(idx=idx, w=w, loss=ce["loss"], dtable=p["dtable"], g=g, lb=lb, nb=nb)


def test_fp32_step_against_autograd():
    T, D, F, E, V = 150, 64, 96, 4, 333
    say(f"model step fp32 T{T} D{D} F{F} E{E} V{V}")
    p = model(T, D, F, E, V, torch.float32, 3)
    r = step(p)
    torch.cuda.synchronize()
    leaf = {n: p[n].cpu().double().requires_grad_() for n in ("table", "ln_w", "ln_b", "out_w", "out_b", "W1", "W3", "W2")}

    def norm(v, w, b):
        d = v - v.mean(1, keepdim=True)
        return d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * w + b

    x = leaf["table"][p["ids"].cpu().long()] * D ** 0.5
    y = norm(x, leaf["ln_w"], leaf["ln_b"])
    ffn = lambda v, a, c, b: (torch.nn.functional.silu(v @ a) * (v @ c)) @ b  # noqa: E731
    idx, w = r["idx"].cpu().long(), r["w"].cpu().double()      # the routing is given: no gradient through it
    each = torch.stack([ffn(y, leaf["W1"][e], leaf["W3"][e], leaf["W2"][e]) for e in range(E)], 1)
    out = x + (each.gather(1, idx[:, :, None].expand(-1, -1, D)) * w[:, :, None]).sum(1)
    z = norm(out, leaf["out_w"], leaf["out_b"]) @ leaf["table"].t()
    t = p["targets"].cpu().long()
    loss = torch.nn.functional.cross_entropy(z, t.clamp(min=-1), ignore_index=-1, reduction="none")
    (loss.sum() / T).backward()
    got = {"loss": (r["loss"], loss.detach()), "table": (r["dtable"], leaf["table"].grad), "ln_w": (r["nb"]["dweight"], leaf["ln_w"].grad),
           "ln_b": (r["nb"]["dbias"], leaf["ln_b"].grad), "out_w": (r["lb"]["dweight"], leaf["out_w"].grad),
           "out_b": (r["lb"]["dbias"], leaf["out_b"].grad)}
    got.update({n: (r["g"]["d" + n], leaf[n].grad) for n in ("W1", "W3", "W2")})
    for name, (a, want) in got.items():
        off = float((a.double().cpu() - want).abs().max())
        assert off <= 1e-4 * float(want.abs().max()), f"{name}: {off:.2e} of {float(want.abs().max()):.2e}"


def test_captured_bf16_step_is_the_eager_step():
    """Captured once and replayed with other tokens and another table, beside the same steps run eagerly."""
    T, D, F, E, V = 1100, 128, 256, 8, 2000
    a = model(T, D, F, E, V, torch.bfloat16, 9)
    step(a)
    torch.cuda.synchronize()
    say("model step captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(a)
    for k in range(4):
        b = model(T, D, F, E, V, torch.bfloat16, 20 + k)
        for name in a:
            if name != "dtable":
                a[name].copy_(b[name])
        graph.replay()
        torch.cuda.synchronize()
        e = step(b)
        torch.cuda.synchronize()
        assert torch.equal(r["loss"], e["loss"]) and torch.equal(r["dtable"], e["dtable"])
        for name in ("dW1", "dW3", "dW2"):
            assert torch.equal(r["g"][name], e["g"][name]), (k, name)
