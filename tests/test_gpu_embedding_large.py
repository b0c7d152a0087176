"""The gradient of tables of many entries."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
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
