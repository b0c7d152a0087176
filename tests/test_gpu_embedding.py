"""Embedding lookup and its table's gradient against 64 bits.

y is one product in fp32 and one rounding: u and half a step of the type.  A gradient's entry is a sum of n rows in fp32
((n + 2) u of the sum of magnitudes, n at most the tokens of the entry), times scale, plus what was there, rounded once.
"""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from vocab_util import HALF, U, within

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def tokens(T, V, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":                                     # every token the same
        ids = torch.full((T,), V // 2, device="cuda")
    elif kind == "often":                                 # the first entries most often, a few outside the table
        ids = ((V + 1.0) ** torch.rand(T, generator=g, device="cuda")).long() - 1
        drop = torch.rand(T, generator=g, device="cuda")
        ids = torch.where(drop < 0.03, torch.full_like(ids, -1), ids)
        ids = torch.where(drop > 0.97, torch.full_like(ids, V), ids)
    else:
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    return ids.int()


SIZES = [(1, 1, 1), (1, 768, 50), (5, 3, 1), (64, 8, 17), (65, 20, 5), (128, 768, 2), (513, 33, 1000), (1000, 1024, 300),
         (4097, 129, 5000), (9000, 96, 40), (300, 64, 20000),
         # beside the most tokens that take one launch
         (1023, 8, 3000), (1024, 12, 5000), (1024, 33, 1000), (1025, 1, 1), (1025, 8, 17), (1100, 20, 5), (1500, 768, 50),
         (2000, 1024, 300), (3000, 64, 20000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_lookup(T, D, V, dtype):
    say(f"embedding T{T} D{D} V{V} {dtype}")
    dt = TYPES[dtype]
    table = torch.randn(V, D, device="cuda").to(dt)
    ids = tokens(T, V, T, "often")
    for scale in (1.0, D ** 0.5):
        got = gg.embedding(ids, table, scale=scale)
        torch.cuda.synchronize()
        inside = (ids >= 0) & (ids < V)
        s = torch.tensor(scale, dtype=torch.float32).double().item()
        want = table[ids.long().clamp(0, V - 1)].double() * s * inside[:, None]
        within(got, want, want.abs() * (HALF[dt] * 1.01 + U), "y")
        if scale == 1.0:
            assert torch.equal(got.double(), want)


@pytest.mark.parametrize("kind", ["even", "often", "one"])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_gradient(T, D, V, dtype, grad, kind):
    say(f"embedding backward T{T} D{D} V{V} {dtype} {grad} {kind}")
    dt, gdt = TYPES[dtype], TYPES[grad]
    dy = torch.randn(T, D, device="cuda").to(dt)
    ids = tokens(T, V, T + 1, kind)
    inside = (ids >= 0) & (ids < V)
    at = ids.long().clamp(0, V - 1)
    scale = 1.5
    rows = dy.double() * inside[:, None]
    sums = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, rows)
    mags = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs())
    n = torch.bincount(at[inside], minlength=V)[:, None].double()
    far = scale * mags * (n + 2) * U
    got = gg.embedding_backward(ids, dy, V, scale=scale, grad_dtype=gdt)
    torch.cuda.synchronize()
    want = scale * sums
    within(got, want, far + HALF[gdt] * (want.abs() + far), "dtable")
    assert torch.equal(got, gg.embedding_backward(ids, dy, V, scale=scale, grad_dtype=gdt))
    base = torch.randn(V, D, device="cuda").to(gdt)
    out = base.clone()
    r = gg.embedding_backward(ids, dy, V, scale=scale, out=out, accumulate=True)
    assert r is out
    want = base.double() + scale * sums
    within(out, want, far + U * want.abs() + HALF[gdt] * (want.abs() + far), "added")
    empty = (n == 0)[:, 0]
    assert torch.equal(out[empty], base[empty])
