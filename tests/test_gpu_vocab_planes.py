"""The losses over fp32 operands, whose products are six of three bf16 planes each: what each of the six adds is seen.

With e = 2^-10, planes of 1 + a e + b e^2 (a, b = 1 or -1) are 1, a e and b e^2: half a step of bf16 below 1 is 2^-9, and e and e^2
are powers of two with 1 / e and e far from each other's rounding.  Sums over pairs (1 + a e + b e^2)(1 + c e + d e^2) - 1 leave
(a + c) e + (b + d + a c) e^2 + (a d + b c) e^3 + b d e^4 each: of the six products the first (of the leading planes) cancels, two
make e and three e^2, and those left out are at most 2 e^3 + e^4.  All partial sums are multiples of e^2 below 2^4, numbers of 24 bits:
adding them rounds nothing, in any order.  So a sum of n pairs is off by at most n (2 e^3 + e^4), a thousandth of what one product
in the least place adds (n e^2).

The give-back of bf16: with an lse of 30 a row's dz is -g at its target and g e^-30 elsewhere, so dh is -g times the target's row of
the table to 2^-20, rounded once; without what rounding g to bf16 took it would be off by up to two roundings."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from vocab_util import U, gradients64, log_sum, within

pytestmark = pytest.mark.gpu
E = 2.0 ** -10
LEFT = 2 * E ** 3 + E ** 4


def signs(*shape, g):
    return torch.randint(0, 2, shape, generator=g, device=g.device).float() * 2 - 1


def generator(device, seed):
    return torch.Generator(device=device).manual_seed(seed)


def for_logits(T, D, V, device):
    """(h, W, how far off a logit may be)."""
    g = generator(device, T)
    n = D // 2
    s = 2.0 ** (16 - (n - 1).bit_length())
    h, W = torch.full((T, D), s, device=device), torch.full((V, D), -1.0, device=device)
    h[:, ::2] *= 1 + signs(T, 1, g=g) * E + signs(T, 1, g=g) * E * E
    W[:, ::2] = 1 + signs(V, 1, g=g) * E + signs(V, 1, g=g) * E * E
    return h, W, s * n * LEFT


def for_dh(T, D, V, device):
    """(the losses' gradient w, W, how far off dh may be): dz is w but for 0 at the target."""
    g = generator(device, T + 1)
    W = torch.full((V, D), -1.0, device=device)
    W[::2] = 1 + signs(1, D, g=g) * E + signs(1, D, g=g) * E * E
    W[1:8:2] = 0                                            # four leading planes that nothing cancels, for dz's other planes
    return 1 + signs(T, g=g) * E + signs(T, g=g) * E * E, W, (V + 1) // 2 * LEFT + 16 * U


def for_dW(T, D, V, a, b, device):
    """(w, h, how far off dW may be)."""
    g = generator(device, T + 2)
    h, w = torch.ones(T, D, device=device), torch.full((T,), -1.0, device=device)
    h[::2] = 1 + signs(1, D, g=g) * E + signs(1, D, g=g) * E * E
    w[::2] = 1 + a * E + b * E * E
    w[1:8:2] = -1 + E - E * E                               # and pairs of which each has all planes
    return w, h, (T + 1) // 2 * LEFT + 16 * U


# tiles of 128 rows (not listed, D no multiple of 4), of 256 (not listed, listed); one, two and four K steps and more, odd ones
SIZES = [(300, 130, 700), (270, 34, 1025), (490, 258, 3000), (600, 128, 900), (1500, 96, 1026), (2100, 256, 520), (700, 1024, 300)]


@pytest.mark.parametrize("T,D,V", SIZES)
def test_logits(T, D, V):
    """loss and lse of the forward, dh and dW of the backward's logits: z from 0 to 256, of which a product of e^2 is 1 / 16."""
    say(f"planes of the logits T{T} D{D} V{V}")
    h, W, most = for_logits(T, D, V, "cuda")
    g = generator("cuda", T + 4)
    target = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    z = h.double() @ W.double().t().contiguous()
    off = torch.full_like(z, most)
    lse, slack = log_sum(z, off, 1.0)
    at = z.gather(1, target.long()[:, None])[:, 0]
    assert float(z.abs().max()) > 50
    f = gg.cross_entropy(h, W, target)
    torch.cuda.synchronize()
    within(f["lse"], lse, slack, "lse")
    within(f["loss"], lse - at, slack + off[:, 0] + 4 * U * z.abs().amax(1), "loss")
    w = torch.rand(T, generator=g, device="cuda") + 0.5
    lse = lse.float()
    b = gg.cross_entropy_backward(h, W, target, lse, w)
    torch.cuda.synchronize()
    hot = torch.zeros_like(z).scatter_(1, target.long()[:, None], 1.0)
    (dh, x), (dW, y) = gradients64(h, W, z, off, lambda p: p - hot, 1.0, lse, w, torch.ones_like(target, dtype=torch.bool), W.dtype)
    within(b["dh"], dh, x, "dh")
    within(b["dW"], dW, y, "dW")


@pytest.mark.parametrize("T,D,V", SIZES)
def test_dh(T, D, V):
    """h = 0 and lse = 0: dz is g but for 0 at the target, all of it known."""
    say(f"planes of dh T{T} D{D} V{V}")
    w, W, most = for_dh(T, D, V, "cuda")
    target = torch.randint(0, V, (T,), generator=generator("cuda", T + 5), device="cuda").int()
    b = gg.cross_entropy_backward(torch.zeros(T, D, device="cuda"), W, target, torch.zeros(T, device="cuda"), w, wanted=("dh",))
    torch.cuda.synchronize()
    dz = w.double()[:, None].expand(T, V).scatter(1, target.long()[:, None], 0.0)
    within(b["dh"], dz @ W.double(), torch.full((T, D), most, dtype=torch.float64, device="cuda"), "dh")


# and few rows, whose dW is made by the tiles of planes
@pytest.mark.parametrize("T,D,V", SIZES + [(200, 64, 9000), (384, 256, 2000)])
def test_dW(T, D, V):
    """A table of zeros and lse = 0: dz is g but for 0 at the target; rows by pairs."""
    say(f"planes of dW T{T} D{D} V{V}")
    for a, b in ((1, 1), (1, -1), (-1, 1)):
        w, h, most = for_dW(T, D, V, a, b, "cuda")
        target = torch.randint(0, V, (T,), generator=generator("cuda", T + 6), device="cuda").int()
        got = gg.cross_entropy_backward(h, torch.zeros(V, D, device="cuda"), target, torch.zeros(T, device="cuda"), w, wanted=("dW",))["dW"]
        torch.cuda.synchronize()
        dz = w.double()[:, None].expand(T, V).scatter(1, target.long()[:, None], 0.0)
        within(got, dz.t().contiguous() @ h.double(), torch.full((V, D), most, dtype=torch.float64, device="cuda"), "dW")


# tiles of 128 rows, of 256 (not listed, listed), of 128 listed
@pytest.mark.parametrize("kind", ["loss", "distill"])
@pytest.mark.parametrize("T,D,V", [(300, 36, 700), (600, 160, 70000), (900, 128, 16400), (1300, 128, 900), (1500, 96, 1025)])
def test_what_rounding_takes_from_a_rows_largest_entry_is_given_back(T, D, V, kind):
    say(f"give-back {kind} T{T} D{D} V{V}")
    g = generator("cuda", T + 3)
    W = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    h = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    target = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    w = (torch.rand(T, generator=g, device="cuda") + 1) * signs(T, g=g)
    lse = torch.full((T,), 30.0, device="cuda")
    if kind == "loss":
        b = gg.cross_entropy_backward(h, W, target, lse, w, wanted=("dh",))
    else:
        ids = target[:, None].expand(T, 2).contiguous()       # one entry twice
        b = gg.distillation_backward(h, W, ids, torch.randn(T, 2, generator=g, device="cuda"), torch.zeros(T, 2, device="cuda"), lse, w, wanted=("dh",))
    torch.cuda.synchronize()
    want = -w.double()[:, None] * W[target.long()].double()
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - 8)
    # the others' share: V e^-30 g of the table's values, at most 6
    within(b["dh"], want, half + want.abs() * 2.0 ** -20 + 12 * V * 1e-13, "dh")
