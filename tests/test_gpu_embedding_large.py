"""The gradient of tables of many entries."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_embedding import tokens
from vocab_util import HALF, U, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 1100])
def test_a_row_of_a_workgroups_own_for_each_of_the_most_entries(T):
    """2^24 entries of more columns than a workgroup takes of several: a workgroup each would be 2^32 threads."""
    D, V = 1025, 1 << 24
    say(f"embedding backward T{T} D{D} V{V}")
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    ids[0], ids[1], ids[2] = V - 1, 0, V - 1
    dy = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    out = torch.full((V, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gg.embedding_backward(ids, dy, V, out=out)
    torch.cuda.synchronize()
    entries, at = ids.long().unique(return_inverse=True)
    n = len(entries)
    want = torch.zeros(n, D, dtype=torch.float64, device="cuda").index_add_(0, at, dy.double())
    mags = torch.zeros(n, D, dtype=torch.float64, device="cuda").index_add_(0, at, dy.double().abs())
    far = mags * (at.bincount()[:, None] + 2) * U
    within(out[entries], want, far + HALF[torch.bfloat16] * (want.abs() + far), "dtable")
    rows = sum(int((out[v:v + (1 << 20)] != 0).any(1).sum()) for v in range(0, V, 1 << 20))
    assert rows == n, "entries without a token are zeros"


# more entries than 256 for each of 256 sorting workgroups, than 1024 for each, for each of 512, of 1024
@pytest.mark.parametrize("kind", ["even", "often", "one"])
@pytest.mark.parametrize("T,V", [(1100, 65536), (1100, 65537), (40000, 100003), (5000, 262144), (5000, 262145), (30000, 600000), (3000, 1 << 24)])
def test_gradient_of_large_tables(T, V, kind):
    D = 24
    say(f"embedding backward T{T} D{D} V{V} {kind}")
    ids = tokens(T, V, T, kind)
    dy = torch.randn(T, D, device="cuda").bfloat16()
    got = gg.embedding_backward(ids, dy, V, scale=0.5, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    inside = (ids >= 0) & (ids < V)
    at, rows = ids.long().clamp(0, V - 1), dy.double() * inside[:, None]
    sums = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, rows)
    mags = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs())
    n = torch.bincount(at[inside], minlength=V)[:, None].double()
    far = 0.5 * mags * (n + 2) * U
    within(got, 0.5 * sums, far + HALF[torch.float32] * (0.5 * sums.abs() + far), "dtable")
    assert torch.equal(got, gg.embedding_backward(ids, dy, V, scale=0.5, grad_dtype=torch.float32))
