"""Cross entropy and distillation over a vocabulary, forward and backward, against 64 bits on the same inputs."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from vocab_util import distill64, gradients64, loss64, product, teacher64, within

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# (T, D, V): single tokens and entries, tile edges of both, widths that are no K step, rows enough to be listed
SIZES = [(1, 64, 1), (1, 768, 1000), (3, 1, 5), (2, 8, 255), (127, 33, 256), (128, 32, 257), (129, 200, 511), (300, 96, 513),
         (700, 64, 5000), (1023, 40, 300), (1024, 64, 300), (1500, 96, 1025), (2500, 130, 70),
         # few rows: one and two blocks of 32, several tiles, columns past a tile, entries past a step
         (32, 136, 129), (33, 72, 1000), (64, 768, 3001), (65, 264, 40), (255, 516, 1100), (256, 40, 17), (257, 64, 500),
         (3, 1024, 1500), (32, 2048, 700), (5, 72, 33000), (1, 1024, 32700), (40, 136, 33001), (65, 264, 16500), (200, 64, 9000),
         # many rows on whole tiles, the last of one row, several tiles a workgroup
         (1025, 128, 2000), (3000, 256, 9000), (4353, 384, 300), (400, 256, 32769), (900, 128, 16400),
         # gradients: whole tiles and a rest shared out, steps shared out evenly (dW, dh)
         (1400, 1100, 14000), (2600, 1001, 9400), (9400, 1000, 2600),
         # and dW of a round of whole tiles and one of halves
         (300, 600, 27000)]


def inputs(T, D, V, dtype, masked, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    W = (n(V, D) * D ** -0.5).to(TYPES[dtype])
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    h = (n(T, D) * 2 + 3 * W[target].float()).to(TYPES[dtype])
    keep = torch.rand(T, generator=g, device="cuda") >= masked
    target = torch.where(keep, target, torch.full_like(target, -100)).int()
    return h, W, target, n(T)


def teacher(T, V, K, seed, masked=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda")       # the same id twice, where it happens
    logits = torch.randn(T, K, generator=g, device="cuda") * 3
    drop = torch.rand(T, K, generator=g, device="cuda")
    ids = torch.where(drop < 0.05, torch.full_like(ids, -1), ids)
    ids = torch.where((drop > 0.05) & (drop < 0.1), torch.full_like(ids, V), ids)
    logits = torch.where((drop > 0.1) & (drop < 0.15), torch.full_like(logits, -float("inf")), logits)
    row = torch.rand(T, generator=g, device="cuda") < masked
    return torch.where(row[:, None], torch.full_like(ids, -7), ids).int(), logits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_cross_entropy(T, D, V, dtype):
    say(f"cross entropy T{T} D{D} V{V} {dtype}")
    h, W, target, _ = inputs(T, D, V, dtype, 0.3 if T > 1 else 0.0, T + D)
    got = gg.cross_entropy(h, W, target)
    torch.cuda.synchronize()
    loss, far, lse, slack = loss64(h, W, target)
    within(got["lse"], lse, slack, "lse")
    within(got["loss"], loss, far, "loss")


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_cross_entropy_backward(T, D, V, dtype, grad):
    say(f"cross entropy backward T{T} D{D} V{V} {dtype} {grad}")
    h, W, target, g = inputs(T, D, V, dtype, 0.3 if T > 1 else 0.0, T + D + 1)
    z, off = product(h, W, W.dtype)
    live = (target >= 0) & (target < V)
    lse = (torch.logsumexp(z, 1) * live).float()
    gdt = TYPES[grad]
    got = gg.cross_entropy_backward(h, W, target, lse, g, grad_dtype=gdt)
    torch.cuda.synchronize()
    hot = torch.zeros_like(z).scatter_(1, target.long().clamp(0, V - 1)[:, None], 1.0)
    (dh, a), (dW, b) = gradients64(h, W, z, off, lambda p: p - hot, 1.0, lse, g, live, gdt)
    assert got["dW"].dtype == gdt and got["dh"].dtype == W.dtype
    within(got["dh"], dh, a, "dh")
    within(got["dW"], dW, b, "dW")


@pytest.mark.parametrize("K,tau", [(1, 1.0), (7, 0.5), (64, 2.0), (65, 1.0), (256, 4.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", SIZES[1::3])
def test_distillation(T, D, V, dtype, K, tau):
    say(f"distillation T{T} D{D} V{V} K{K} {dtype}")
    h, W, _, g = inputs(T, D, V, dtype, 0.0, T + D + 2)
    ids, logits = teacher(T, V, K, T + K)
    got = gg.distillation(h, W, ids, logits, temperature=tau)
    torch.cuda.synchronize()
    loss, far, lse, slack, z, zoff = distill64(h, W, ids, logits, tau)
    within(got["lse"], lse, slack, "lse")
    within(got["z"], z, zoff, "z")
    within(got["loss"], loss, far, "loss")

    say("its backward")
    zf, off = product(h, W, W.dtype)
    count, q, _ = teacher64(ids, logits, V, tau)
    live = count.any(1)
    lse = (torch.logsumexp(zf / tau, 1) * live).float()
    back = gg.distillation_backward(h, W, ids, logits, got["z"], lse, g, temperature=tau, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    want = torch.zeros_like(zf).scatter_add_(1, ids.long().clamp(0, V - 1), q)
    # the teacher's q is off by up to (16 + K + its exponent) u: at entries that ids name, in units of g / tau
    (dh, a), (dW, b) = gradients64(h, W, zf, off, lambda p: p - want, tau, lse, g, live, torch.float32)
    w = (g.double().abs() / tau * live)[:, None] * want * 2.0 ** -24 * (24 + 2 * K + 2 * logits.double().nan_to_num(neginf=0).abs().amax(1, keepdim=True) / tau)
    within(back["dh"], dh, a + w @ W.double().abs(), "dh")
    within(back["dW"], dW, b + w.t().contiguous() @ h.double().abs(), "dW")
