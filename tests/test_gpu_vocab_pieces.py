"""Gradients of the losses whose dz is made in several pieces of the vocabulary, against 64 bits.

The table is zero but for the entries beside the pieces' borders and at both ends, which the targets and the teachers' entries
name: sums over the vocabulary have these terms alone (adding zeros rounds nothing), and all other entries' gradients are
alike.  So the formulas are worked out for a few hundred entries and one that stands for the rest."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_vocab_loss import TYPES
from vocab_util import gradients64, product, teacher64, within

pytestmark = pytest.mark.gpu


def borders(T, V, each):
    """The first entries of the pieces: whole tiles of 256 entries, as even as they can be, of 2 GiB of dz at most."""
    tiles, most = -(-V // 256), (1 << 31) // (T * each) // 256
    pieces = -(-tiles // most)
    assert pieces > 1
    piece = -(-tiles // pieces) * 256
    return list(range(0, V, piece))


def check(T, D, V, dtype, grad, kind, each):
    say(f"pieces {kind} T{T} D{D} V{V} {dtype} {grad}")
    g = torch.Generator(device="cuda").manual_seed(T)
    dt, gdt = TYPES[dtype], TYPES[grad]
    entries = torch.cat([torch.arange(max(0, b - 70), min(V, b + 70)) for b in [*borders(T, V, each), V]]).unique().cuda()
    n = len(entries)
    few = torch.cat([(torch.randn(n, D, generator=g, device="cuda") * D ** -0.5).to(dt), torch.zeros(1, D, dtype=dt, device="cuda")])
    W = torch.zeros(V, D, dtype=dt, device="cuda")
    W[entries] = few[:-1]
    h = torch.randn(T, D, generator=g, device="cuda").to(dt)
    w = torch.randn(T, generator=g, device="cuda")
    tau = 1.0 if kind == "loss" else 2.0
    z, off = product(h, few, dt)
    lse = torch.logsumexp(torch.cat([z[:, :-1] / tau, torch.full_like(z[:, :1], V - n).log()], 1), 1)

    def some(*shape):                                    # places among the entries, a few outside the table
        return torch.randint(-n // 20, n, shape, generator=g, device="cuda").clamp(min=-1)

    names = torch.cat([entries, torch.tensor([-1], device="cuda")]).int()
    more = torch.zeros_like(z)
    if kind == "loss":
        at = some(T)
        live = at >= 0
        want = torch.zeros_like(z).scatter_(1, at.clamp(min=0)[:, None], 1.0)
        lse = (lse * live).float()
        b = gg.cross_entropy_backward(h, W, names[at], lse, w, grad_dtype=gdt)
    else:
        K = 5
        at = some(T, K)
        at[:, 1] = at[:, 0]                              # one entry twice
        at[::11] = -1
        logits = torch.randn(T, K, generator=g, device="cuda")
        count, q, _ = teacher64(at, logits, V, tau)
        live = count.any(1)
        want = torch.zeros_like(z).scatter_add_(1, at.clamp(min=0), q)
        lse = (lse * live).float()
        f = gg.distillation(h, W, names[at], logits, temperature=tau)
        b = gg.distillation_backward(h, W, names[at], logits, f["z"], lse, w, temperature=tau, grad_dtype=gdt)
        # the teacher's q: off by up to (24 + 2 K + its exponent) u
        more = (w.double().abs() / tau * live)[:, None] * want * 2.0 ** -24 * (24 + 2 * K + logits.double().abs().amax(1, keepdim=True))
    torch.cuda.synchronize()
    (dh, x), (dW, y) = gradients64(h, few, z, off, lambda p: p - want, tau, lse, w, live, gdt)
    within(b["dh"], dh, x + more @ few.double().abs(), "dh")
    y = y + more.t().contiguous() @ h.double().abs()
    within(b["dW"][entries], dW[:-1], y[:-1], "dW")
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[entries] = False
    for v in range(0, V, 1 << 20):
        c = slice(v, v + (1 << 20))
        over = (b["dW"][c].double() - dW[-1]).abs() - y[-1]
        assert float(torch.where(rest[c, None], over, torch.full_like(over, -1.0)).max()) <= 0, f"dW of an entry that nothing names, from {v}"


@pytest.mark.parametrize("kind", ["loss", "distill"])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,D,V", [(64, 8, 9_000_001), (40, 24, 1 << 24)])
def test_few_rows_of_very_many_entries(T, D, V, dtype, grad, kind):
    check(T, D, V, dtype, grad, kind, 4)


# tiles of 256 rows (listed; in three pieces), of 128 listed, of 128 not listed; of fp32 planes the same but for the second, whose rows are padded to whole tiles
@pytest.mark.parametrize("kind", ["loss", "distill"])
@pytest.mark.parametrize("T,D,V,dtype,grad", [(70000, 128, 20000, "bf16", "bf16"), (50000, 128, 50001, "bf16", "f32"), (60000, 96, 18433, "bf16", "bf16"),
                                              (300, 36, 3_700_001, "bf16", "bf16"), (300, 33, 3_700_001, "bf16", "f32"),
                                              (30000, 64, 20000, "f32", "f32"), (20000, 40, 40001, "f32", "f32"), (300, 33, 1_300_001, "f32", "f32")])
def test_many_rows(T, D, V, dtype, grad, kind):
    check(T, D, V, dtype, grad, kind, 2 if dtype == "bf16" else 6)
