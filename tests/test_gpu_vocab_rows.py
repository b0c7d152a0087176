"""Cross entropy and distillation of more rows than one launch has threads for: 2^32 in a grid are 2^24 rows of a workgroup
or 2^26 of a wavefront each.  Few entries, short rows: every row is compared with the formulas in 64 bits."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from vocab_util import distill64, gradients64, product, teacher64, within

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
