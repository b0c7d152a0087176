"""Embedding, cross entropy and distillation: what the C entry points and the binding refuse on the host, and the sizes of
their workspaces (no GPU needed; no pointer here is dereferenced)."""
import pytest
import torch

gg = pytest.importorskip("grouped_gemm_permute_amd")
from grouped_gemm_permute_amd import _lib as L  # noqa: E402

FAKE = 0x7F0000000000
BAD, UNSUPPORTED, OK = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_OK
INF, NAN = float("inf"), float("nan")


def call(name, defaults, over):
    a = dict(defaults)
    assert set(over) <= set(a), over
    a.update(over)
    return getattr(L.lib(), name)(*a.values(), None)


LOOKUP = dict(ids=FAKE, table=FAKE, y=FAKE, T=16, D=64, V=100, scale=1.0, dt=L.MOE_BF16)
LOOKUP_BACK = dict(ids=FAKE, dy=FAKE, dtable=FAKE, T=16, D=64, V=100, scale=1.0, add=0, dt=L.MOE_BF16, gdt=L.MOE_F32, ws=FAKE, n=1 << 30)
LOSS = dict(h=FAKE, W=FAKE, t=FAKE, loss=FAKE, lse=FAKE, T=16, D=64, V=100, dt=L.MOE_BF16, ws=FAKE, n=1 << 40)
LOSS_BACK = dict(h=FAKE, W=FAKE, t=FAKE, lse=FAKE, g=FAKE, dh=FAKE, dW=FAKE, T=16, D=64, V=100, dt=L.MOE_BF16, gdt=L.MOE_F32, ws=FAKE, n=1 << 40)
DIST = dict(h=FAKE, W=FAKE, ids=FAKE, q=FAKE, loss=FAKE, lse=FAKE, z=FAKE, T=16, D=64, V=100, K=4, tau=1.0, dt=L.MOE_BF16, ws=FAKE, n=1 << 40)
DIST_BACK = dict(h=FAKE, W=FAKE, ids=FAKE, q=FAKE, z=FAKE, lse=FAKE, g=FAKE, dh=FAKE, dW=FAKE, T=16, D=64, V=100, K=4, tau=1.0,
                 dt=L.MOE_BF16, gdt=L.MOE_F32, ws=FAKE, n=1 << 40)


@pytest.mark.parametrize("over,status", [
    (dict(ids=None), BAD), (dict(table=None), BAD), (dict(y=None), BAD), (dict(table=FAKE + 8), BAD), (dict(y=FAKE + 2), BAD),
    (dict(ids=FAKE + 2), BAD), (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(D=0), BAD), (dict(V=0), BAD), (dict(dt=2), BAD),
    (dict(scale=INF), BAD), (dict(scale=NAN), BAD), (dict(D=16385), UNSUPPORTED), (dict(V=(1 << 24) + 1), UNSUPPORTED),
    (dict(T=(1 << 26) + 1), UNSUPPORTED), (dict(T=0, ids=None, table=None, y=None), OK),
])
def test_lookup_refusals(over, status):
    assert call("moe_embedding_forward", LOOKUP, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(ids=None), BAD), (dict(dy=None), BAD), (dict(dtable=None), BAD), (dict(dtable=None, T=0), BAD), (dict(ws=None), BAD),
    (dict(ws=FAKE + 128), BAD), (dict(dy=FAKE + 8), BAD), (dict(dtable=FAKE + 8), BAD), (dict(ids=FAKE + 1), BAD),
    (dict(dt=L.MOE_F32, gdt=L.MOE_BF16), BAD), (dict(gdt=5), BAD), (dict(dt=5), BAD), (dict(scale=NAN), BAD), (dict(T=-1), BAD),
    (dict(V=0), BAD), (dict(D=0), BAD), (dict(n=100), L.MOE_ERR_WORKSPACE), (dict(D=20000), UNSUPPORTED),
    (dict(T=0, add=1, ids=None, dy=None), OK),
])
def test_lookup_backward_refusals(over, status):
    assert call("moe_embedding_backward", LOOKUP_BACK, over) == status


SHARED = [
    (dict(h=None), BAD), (dict(W=None), BAD), (dict(lse=None), BAD), (dict(h=FAKE + 8), BAD), (dict(W=FAKE + 4), BAD),
    (dict(lse=FAKE + 2), BAD), (dict(T=-1), BAD), (dict(D=0), BAD), (dict(V=0), BAD), (dict(V=-3), BAD), (dict(dt=3), BAD),
    (dict(ws=None), BAD), (dict(ws=FAKE + 64), BAD), (dict(n=64), L.MOE_ERR_WORKSPACE), (dict(D=16385), UNSUPPORTED),
    (dict(V=(1 << 24) + 1), UNSUPPORTED), (dict(T=(1 << 28) + 1), UNSUPPORTED), (dict(T=1 << 24, V=1 << 24), UNSUPPORTED),
    (dict(T=1 << 27, D=16384, V=1), UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(t=None), BAD), (dict(t=FAKE + 2), BAD), (dict(loss=None), BAD), (dict(loss=FAKE + 2), BAD),
    (dict(T=0, h=None, W=None, t=None, loss=None, lse=None, ws=None), OK),
])
def test_loss_refusals(over, status):
    assert call("moe_cross_entropy_forward", LOSS, over) == status


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(t=None), BAD), (dict(g=None), BAD), (dict(g=FAKE + 2), BAD), (dict(dh=None, dW=None), BAD), (dict(dh=FAKE + 8), BAD),
    (dict(dW=FAKE + 8), BAD), (dict(gdt=4), BAD), (dict(dt=L.MOE_F32, gdt=L.MOE_BF16), BAD),
    (dict(T=0, h=None, W=None, t=None, lse=None, g=None, dh=None, dW=None, ws=None), OK),
])
def test_loss_backward_refusals(over, status):
    assert call("moe_cross_entropy_backward", LOSS_BACK, over) == status


TEACHER = [(dict(ids=None), BAD), (dict(q=None), BAD), (dict(z=None), BAD), (dict(ids=FAKE + 2), BAD), (dict(q=FAKE + 2), BAD),
           (dict(z=FAKE + 1), BAD), (dict(K=0), BAD), (dict(K=-1), BAD), (dict(K=257), UNSUPPORTED), (dict(tau=0.0), BAD),
           (dict(tau=-1.0), BAD), (dict(tau=INF), BAD), (dict(tau=NAN), BAD), (dict(tau=1e-39), BAD)]


@pytest.mark.parametrize("over,status", SHARED + TEACHER + [(dict(loss=None), BAD)])
def test_distillation_refusals(over, status):
    assert call("moe_distillation_forward", DIST, over) == status


@pytest.mark.parametrize("over,status", SHARED + TEACHER + [(dict(g=None), BAD), (dict(dh=None, dW=None), BAD), (dict(gdt=9), BAD)])
def test_distillation_backward_refusals(over, status):
    assert call("moe_distillation_backward", DIST_BACK, over) == status


def test_workspace_sizes():
    bf16, f32 = torch.bfloat16, torch.float32
    loss, dist = gg.cross_entropy_workspace_size, gg.distillation_workspace_size
    assert loss(0, 64, 100, bf16, True) == 0 and dist(0, 64, 100, 4, f32, False) == 0
    assert loss(1, 16385, 100, bf16, False) == 0 and dist(1, 64, 100, 257, bf16, False) == 0 and dist(1, 64, 100, 0, bf16, True) == 0
    # the forward keeps 8 bytes for 256 entries of a row, not the logits
    assert loss(32768, 768, 65536, bf16, False) < 32768 * (8 * 256 + 2 * 768 + 64) + (1 << 20)
    # the backward keeps one piece of dz, 2 GiB of it or 256 entries, whatever the vocabulary
    assert loss(32768, 768, 1 << 20, bf16, True) < (2 << 30) + (1 << 29)
    assert loss(32768, 768, 65536, bf16, True) > 1 << 30
    assert loss(1, 768, 50001, bf16, True) < 4 << 20
    # fp32 operands are copied in three planes of bf16, those of few rows are not
    assert loss(4096, 768, 50000, f32, False) > 3 * 2 * 768 * 50000
    assert loss(16, 768, 50000, f32, False) < 1 << 20
    assert dist(2000, 64, 100, 4, bf16, False) > 0
    e = gg.embedding_backward_workspace_size
    assert e(0, 64, 100) > 0 and e(1, 20000, 10) == 0 and e(-1, 64, 10) == 0
    assert e(32768, 768, 65536) < 32768 * (4 + 768 * 8 // 32) + 2 * 4 * 65536 + 4096
    with pytest.raises(TypeError, match="dtype"):
        loss(4, 64, 100, torch.float16, True)


def test_binding_refusals():
    bf = torch.bfloat16
    ids, W, h = torch.zeros(8, dtype=torch.int32), torch.zeros(100, 64, dtype=bf), torch.zeros(8, 64, dtype=bf)
    s = torch.zeros(8)
    k, q = torch.zeros(8, 4, dtype=torch.int32), torch.zeros(8, 4)
    checks = [
        (ValueError, "GPU", lambda: gg.embedding(ids, W)),
        (TypeError, "ids", lambda: gg.embedding(ids.long(), W)),
        (ValueError, r"\[T\]", lambda: gg.embedding(ids[None], W)),
        (ValueError, r"\[V,D\]", lambda: gg.embedding(ids, W[0])),
        (ValueError, "contiguous", lambda: gg.embedding(ids, W.t())),
        (TypeError, "dtype", lambda: gg.embedding(ids, W.half())),
        (ValueError, "out", lambda: gg.embedding(ids, W, out=h[:4])),
        (ValueError, "V must be", lambda: gg.embedding(ids, W[:0])),
        (ValueError, "GPU", lambda: gg.embedding_backward(ids, h, 100)),
        (ValueError, "ids", lambda: gg.embedding_backward(ids[:4], h, 100)),
        (ValueError, r"\[T,D\]", lambda: gg.embedding_backward(ids, h[0], 100)),
        (ValueError, "accumulate", lambda: gg.embedding_backward(ids, h, 100, accumulate=True)),
        (TypeError, "gradient", lambda: gg.embedding_backward(ids, h, 100, grad_dtype=torch.float16)),
        (TypeError, "gradient", lambda: gg.embedding_backward(ids, h.float(), 100, grad_dtype=bf)),
        (ValueError, "out", lambda: gg.embedding_backward(ids, h, 100, out=W[:99])),
        (ValueError, "V must be", lambda: gg.embedding_backward(ids, h, 1 << 32)),
        (ValueError, "V must be", lambda: gg.embedding_backward(ids, h, 0)),
        (ValueError, "GPU", lambda: gg.cross_entropy(h, W, ids)),
        (TypeError, "h must be", lambda: gg.cross_entropy(h.float(), W, ids)),
        (ValueError, "h must", lambda: gg.cross_entropy(h[:, :32], W, ids)),
        (TypeError, "targets", lambda: gg.cross_entropy(h, W, ids.long())),
        (ValueError, "targets", lambda: gg.cross_entropy(h, W, ids[:4])),
        (ValueError, "place for dh", lambda: gg.cross_entropy(h, W, ids, out={"dh": h})),
        (ValueError, "GPU", lambda: gg.cross_entropy_backward(h, W, ids, s, s)),
        (TypeError, "dloss", lambda: gg.cross_entropy_backward(h, W, ids, s, s.double())),
        (ValueError, "lse", lambda: gg.cross_entropy_backward(h, W, ids, s[:4], s)),
        (ValueError, "wanted", lambda: gg.cross_entropy_backward(h, W, ids, s, s, wanted=())),
        (ValueError, "wanted", lambda: gg.cross_entropy_backward(h, W, ids, s, s, wanted=("dh", "db"))),
        (ValueError, "place for dW", lambda: gg.cross_entropy_backward(h, W, ids, s, s, wanted=("dh",), out={"dW": W})),
        (TypeError, "dW must be", lambda: gg.cross_entropy_backward(h, W, ids, s, s, grad_dtype=torch.float16)),
        (ValueError, "GPU", lambda: gg.distillation(h, W, k, q)),
        (ValueError, r"\[T,K\]", lambda: gg.distillation(h, W, ids, q)),
        (ValueError, "K must be", lambda: gg.distillation(h, W, k[:, :0], q[:, :0])),
        (ValueError, "logits", lambda: gg.distillation(h, W, k, q[:, :3])),
        (TypeError, "logits", lambda: gg.distillation(h, W, k, q.to(bf))),
        (TypeError, "z must be", lambda: gg.distillation_backward(h, W, k, q, q.double(), s, s)),
        (ValueError, "GPU", lambda: gg.distillation_backward(h, W, k, q, q, s, s)),
    ]
    for kind, text, f in checks:
        with pytest.raises(kind, match=text):
            f()
