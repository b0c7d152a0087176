"""The training step around the layer with the shared expert's matrices stepped too: six Muon steps, three on batches of the
experts' matrices and three on single ones, from the gradients that one backward wrote."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_block_step import BETA, DECAY, LR, block, muon64, step
from test_gpu_muon import U

pytestmark = pytest.mark.gpu
SHARED = ("Ws1", "Ws3", "Ws2")


def block6(*a):
    p = block(*a)
    for name in SHARED:
        p["master_" + name] = p[name].float()
        p["mom_" + name] = torch.zeros(p[name].shape, device="cuda")
    return p


def step6(p):
    r = step(p)
    for name in SHARED:
        bf16 = p[name].dtype == torch.bfloat16
        gg.muon_step(p["master_" + name], r["g"]["d" + name], p["mom_" + name], LR, beta=BETA, weight_decay=DECAY,
                     W_bf16=p[name] if bf16 else None)
    return r


@pytest.mark.parametrize("dtype,T,D,F,E", [(torch.float32, 150, 64, 96, 4), (torch.bfloat16, 700, 128, 256, 8),
                                           (torch.bfloat16, 300, 256, 128, 4)])
def test_shared_experts_matrices(dtype, T, D, F, E):
    say(f"block step, shared expert {dtype} T{T} D{D} F{F} E{E}")
    p = block6(T, D, F, E, dtype, 7)
    before = {n: p[n].float().cpu() for n in SHARED}
    r = step6(p)
    torch.cuda.synchronize()
    for n in SHARED:
        want, most = muon64(before[n][None], r["g"]["d" + n].cpu()[None], U)
        assert ((p["master_" + n].double().cpu()[None] - want).abs() <= most).all(), n
        assert float((p["master_" + n].cpu() - before[n]).abs().max()) > 0
        assert torch.equal(p["mom_" + n], r["g"]["d" + n])
        if dtype == torch.bfloat16:
            assert torch.equal(p[n], p["master_" + n].bfloat16())


def test_captured_and_replayed():
    T, D, F, E = 400, 128, 256, 8
    a, b = block6(T, D, F, E, torch.bfloat16, 9), block6(T, D, F, E, torch.bfloat16, 9)
    step6(block6(T, D, F, E, torch.bfloat16, 9))
    torch.cuda.synchronize()
    say("block step with the shared expert captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step6(a)
    for k in range(4):
        x = block(T, D, F, E, torch.bfloat16, 20 + k)["x"]
        a["x"].copy_(x)
        b["x"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        e = step6(b)
        torch.cuda.synchronize()
        assert torch.equal(r["out"], e["out"])
        for n in ("W1", "W3", "W2", *SHARED):
            assert torch.equal(a[n], b[n]) and torch.equal(a["mom_" + n], b["mom_" + n]), (k, n)
