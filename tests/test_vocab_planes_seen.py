"""That the operands of test_gpu_vocab_planes.py show each of the six products of planes: worked out here in 64 bits from the planes,
with one product left out, or made of another plane, the result is further off than the GPU tests allow (no GPU needed)."""
import pytest
import torch

from test_gpu_vocab_planes import SIZES, for_dh, for_dW, for_logits

SIX = {(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)}


def planes(x):
    p = []
    for _ in range(3):
        p.append(x.bfloat16().float())
        x = x - p[-1]
    assert not x.any()
    return [q.double() for q in p]


def seen(a, b, most, times=2.0):
    """a [M,K], b [N,K]: the six products are near enough, and no five of them, nor six with one of other planes."""
    A, B = planes(a), planes(b)
    every = {(i, j): A[i] @ B[j].t() for i in range(3) for j in range(3)}
    exact = a.double() @ b.double().t()
    assert float((sum(every[p] for p in SIX) - exact).abs().max()) <= most
    for one in SIX - {(0, 0)}:                             # that one cancels; every other test sees it
        five = sum(every[p] for p in SIX - {one})
        assert float((five - exact).abs().max()) > times * most, one
        for i, j in every:
            if (i, j) not in SIX or (i, j) == one:
                continue
            assert float((five + every[i, j] - exact).abs().max()) > times * most, (one, i, j)


@pytest.mark.parametrize("T,D,V", SIZES)
def test_of_the_logits(T, D, V):
    h, W, most = for_logits(T, D, V, "cpu")
    # the loss adds what its exponentials and sums round, 2^-24 of a few times the logits: less than a twentieth of a product
    seen(h, W, most + 2.0 ** -24 * 16 * float((h.double() @ W.double().t()).abs().max()))


@pytest.mark.parametrize("T,D,V", SIZES)
def test_of_dh(T, D, V):
    w, W, most = for_dh(T, D, V, "cpu")
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1))
    dz = w[:, None].expand(T, V).scatter(1, target[:, None], 0.0)
    seen(dz, W.t().contiguous(), most, 1.3)


@pytest.mark.parametrize("T,D,V", SIZES)
def test_of_dW(T, D, V):
    for a, b in ((1, 1), (1, -1), (-1, 1)):
        w, h, most = for_dW(T, D, V, a, b, "cpu")
        target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1))
        dz = w[:, None].expand(T, V).scatter(1, target[:, None], 0.0)
        seen(dz.t().contiguous(), h.t().contiguous(), most)
