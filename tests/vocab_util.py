"""Cross entropy, distillation and embedding in 64 bits, each value with a bound of what the kernels' arithmetic may be off.

u = 2^-24 is half a step of fp32 (relative), HALF[dtype] that of a type.

Products: a sum of n fp32 products (exact for bf16 operands) is off by at most n u times the sum of their magnitudes.
fp32 operands are three bf16 planes: each plane takes 8 bits, so x is off by 2^-24 |x|, the planes beyond the first are
2^-8 |x| and 2^-16 |x|, and the products left out are at most 2 * 2^-24 + 2^-32 of |a b|: 2^-22 |a b| with both, and six
times as many terms are summed.

A row's lse: the logits' own error passes through with weights that sum to 1 (its largest over the row bounds it); the
exponent z c - top is rounded twice (u of each, in units of log 2), the hardware's exp2 and log2 are within 2 u; sums of n terms add
at most 64 u here (32 in a lane, then trees of at most 4 + 16 + the tiles joined by a thread); lse = (top + log2 sum) ln 2 rounds 3 times.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def product(a, b, dtype):
    """(a b^T in 64 bits, its bound) of a [M,K], b [N,K]."""
    a, b = a.double(), b.double()
    z, s = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    n = a.shape[1] + 1
    return z, s * (n * U if dtype == torch.bfloat16 else 6 * n * U + 2.0 ** -22)


def log_sum(z, off, tau):
    """lse of z / tau with the bound of the kernels'."""
    lse = torch.logsumexp(z / tau, 1)
    tiles = math.ceil(z.shape[1] / 256 / 16)
    spread = (z / tau).abs().amax(1)
    return lse, (off / tau).amax(1) + U * (64 + tiles + 4 * spread + 4 * lse.abs())


def loss64(h, W, target):
    """(loss, its bound, lse, its bound); rows without a target 0."""
    V, dt = W.shape[0], W.dtype
    live = (target >= 0) & (target < V)
    h = torch.where(live[:, None], h, torch.zeros_like(h))
    z, off = product(h, W, dt)
    lse, slack = log_sum(z, off, 1.0)
    at = target.long().clamp(0, V - 1)[:, None]
    loss = lse - z.gather(1, at)[:, 0]
    far = slack + off.gather(1, at)[:, 0] + 4 * U * z.abs().amax(1)
    return loss * live, far * live, lse * live, slack * live


def teacher64(ids, logits, V, tau):
    """(entries that count, q, log q) in 64 bits."""
    count = (ids >= 0) & (ids < V) & (logits != -math.inf)
    a = torch.where(count, logits.double() / tau, torch.full_like(logits, -math.inf, dtype=torch.float64))
    some = count.any(1, keepdim=True)
    # the largest off first: at -1e39 even 64 bits would lose the logarithm of the sum
    a = torch.where(some, a - a.max(1, keepdim=True).values, a)
    logq = torch.where(some, a - torch.logsumexp(torch.where(some, a, torch.zeros_like(a)), 1, keepdim=True), torch.zeros_like(a))
    q = torch.where(count, logq.exp(), torch.zeros_like(a))
    return count, q, torch.where(count, logq, torch.zeros_like(a))


def distill64(h, W, ids, logits, tau):
    """(loss, bound, lse, bound, z, bound)."""
    V, dt, K = W.shape[0], W.dtype, ids.shape[1]
    count, q, logq = teacher64(ids, logits, V, tau)
    live = count.any(1)
    z, off = product(h, W, dt)
    lse, slack = log_sum(z, off, tau)
    inside = (ids >= 0) & (ids < V)
    at = ids.long().clamp(0, V - 1)
    zk, zoff = z.gather(1, at) * inside, off.gather(1, at) * inside
    loss = (q * (logq - zk / tau)).sum(1) + lse
    # q: exp and its sum within (8 + K + |exponent|) u; every term q (log q - z / tau) a few roundings more
    mag = (q * (logq.abs() + (zk / tau).abs() + 1)).sum(1)
    far = slack + (q * zoff).sum(1) / tau + U * (16 + 2 * K + 2 * (logq * (q > 0)).abs().amax(1)) * mag + 4 * U * lse.abs()
    return loss * live, far * live, lse * live, slack * live, zk, zoff


def gradients64(h, W, z, off, dz_of, tau, lse, g, live, gdt, rounding=None):
    """((dh, bound), (dW, bound)): dz_of(p) takes the softmax p [T,V] to p - (what a row wants); lse is the given fp32 one."""
    dt = W.dtype
    arg = z / tau - lse.double()[:, None]
    p = arg.exp()
    w = (g.double() / tau * live)[:, None]
    dz = dz_of(p) * w
    # p: the logit's error, the division by tau (two roundings of z / tau), the difference and its product with log2 e, exp2
    rel = off / tau + U * (4 * (z / tau).abs() + 4 * arg.abs() + 8)
    far = w.abs() * p * rel + 4 * U * (dz.abs() + w.abs() * p)
    far = far + dz.abs() * (HALF[dt] if dt == torch.bfloat16 else 2.0 ** -24)
    T, V = z.shape
    hd = torch.where(live[:, None], h, torch.zeros_like(h)).double()
    Wd = W.double()
    one = 1 if dt == torch.bfloat16 else 6
    extra = 0.0 if dt == torch.bfloat16 else 2.0 ** -22
    grown = dz.abs() + far
    dh, dW = dz @ Wd, dz.t().contiguous() @ hd
    dh_far = far @ Wd.abs() + (one * (V + 64) * U + extra) * (grown @ Wd.abs()) + HALF[dt] * dh.abs()
    dW_far = far.t().contiguous() @ hd.abs() + (one * (T + 64) * U + extra) * (grown.t().contiguous() @ hd.abs()) + HALF[gdt] * dW.abs()
    # what is rounded is the value with its error, and the smallest normal numbers have steps of their own
    return (dh, dh_far * 1.01 + 1e-37), (dW, dW_far * 1.01 + 1e-37)


def within(got, want, most, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - most
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} over the bound at {int(over.argmax())}, largest {float(want.abs().max()):.3e}"
