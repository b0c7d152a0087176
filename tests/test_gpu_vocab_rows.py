"""Cross entropy and distillation of more rows than one launch has threads for: 2^32 in a grid are 2^24 rows of a workgroup
or 2^26 of a wavefront each.  Few entries, short rows: every row is compared with the formulas in 64 bits."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from vocab_util import distill64, gradients64, loss64, product, teacher64, within

pytestmark = pytest.mark.gpu


def test_a_teacher_of_more_rows_than_a_launch_takes():
    T, D, V, K = (1 << 26) + 5, 8, 3, 2
    say(f"distillation T{T} D{D} V{V} K{K}")
    g = torch.Generator(device="cuda").manual_seed(2)
    W = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    h = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.randint(-1, V, (T, K), generator=g, device="cuda", dtype=torch.int32)      # rows without an entry among them
    logits = torch.randn(T, K, generator=g, device="cuda")
    f = gg.distillation(h, W, ids, logits, temperature=2.0)
    torch.cuda.synchronize()
    step = 1 << 22
    for t in range(0, T, step):
        c = slice(t, t + step)
        loss, far, lse, slack, z, zoff = distill64(h[c], W, ids[c], logits[c], 2.0)
        within(f["lse"][c], lse, slack, f"lse from row {t}")
        within(f["z"][c], z, zoff, f"z from row {t}")
        within(f["loss"][c], loss, far, f"loss from row {t}")

    say("its backward")
    w = torch.rand(T, generator=g, device="cuda") / T
    b = gg.distillation_backward(h, W, ids, logits, f["z"], f["lse"], w, temperature=2.0, wanted=("dh",))
    torch.cuda.synchronize()
    for t in [*range(0, T, 1 << 23), T - 70000]:            # beside the launches' borders, and the end
        c = slice(max(0, t - 70000), t + 70000)
        z, off = product(h[c], W, W.dtype)
        count, q, _ = teacher64(ids[c], logits[c], V, 2.0)
        want = torch.zeros_like(z).scatter_add_(1, ids[c].long().clamp(0, V - 1), q)
        (dh, a), _ = gradients64(h[c], W, z, off, lambda p: p - want, 2.0, f["lse"][c], w[c], count.any(1), torch.float32)
        # the teacher's q, as in the small tests: off by up to (16 + K + its exponent) u
        more = (w[c].double() / 2)[:, None] * want * 2.0 ** -24 * (24 + 2 * K + logits[c].double().abs().amax(1, keepdim=True))
        within(b["dh"][c], dh, a + more @ W.double().abs(), f"dh about row {t}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [32768, 32769, 36863, 36864, 36865, 100001])
def test_rows_listed_by_counts(T, dtype):
    """About the most rows whose list each workgroup counts by itself, and ends of its chunks of 4096."""
    D, V = 16, 5
    say(f"listed rows T{T} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(T)
    W = torch.randn(V, D, generator=g, device="cuda").to(dtype)
    h = torch.randn(T, D, generator=g, device="cuda").to(dtype)
    target = torch.randint(-2, V + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    target[4096:8192], target[12288:16384] = -1, 2                 # chunks without a row, and of nothing else
    f = gg.cross_entropy(h, W, target)
    loss, far, lse, slack = loss64(h, W, target)
    within(f["loss"], loss, far, "loss")
    within(f["lse"], lse, slack, "lse")
    w = torch.rand(T, generator=g, device="cuda")
    b = gg.cross_entropy_backward(h, W, target, f["lse"], w, grad_dtype=torch.float32)
    z, off = product(h, W, dtype)
    hot = torch.zeros_like(z).scatter_(1, target.long().clamp(0, V - 1)[:, None], 1.0)
    (dh, x), (dW, y) = gradients64(h, W, z, off, lambda p: p - hot, 1.0, f["lse"], w, (target >= 0) & (target < V), torch.float32)
    within(b["dh"], dh, x, "dh")
    within(b["dW"], dW, y, "dW")


def test_a_loss_of_the_most_rows():
    """2^28 rows, the most there may be: a quarter of them without a target, of 2^28 - 3 the last chunk of the list not whole."""
    D, V = 8, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    h = torch.empty(1 << 28, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    target = torch.randint(-1, V, (1 << 28,), generator=g, device="cuda", dtype=torch.int32)
    for T in (1 << 28, (1 << 28) - 3):
        say(f"cross entropy T{T} D{D} V{V}")
        f = gg.cross_entropy(h[:T], W, target[:T])
        torch.cuda.synchronize()
        step = 1 << 22
        for t in range(0, T, step):
            c = slice(t, min(T, t + step))
            loss, far, lse, slack = loss64(h[c], W, target[c])
            within(f["lse"][c], lse, slack, f"lse from row {t}")
            within(f["loss"][c], loss, far, f"loss from row {t}")
