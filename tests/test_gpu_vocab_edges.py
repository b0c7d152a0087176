"""Embedding, cross entropy and distillation where they can go wrong: rows that take no part, values that are no numbers,
borders of the buffers, one call beside or after another, captured calls, sizes past 32 bits."""
import math

import pytest
import torch

import grouped_gemm_permute_amd as gg
from gpu_util import say
from test_gpu_vocab_loss import TYPES, inputs, teacher
from vocab_util import HALF, U, distill64, gradients64, loss64, product, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
# each way through the kernels: few rows (fp32 dW by few rows, by tiles), tiles of 128 and of 256, listed rows on tiles of 128 (D no multiple of 128) and of 256
WAYS = [(40, 64, 700), (150, 72, 700), (200, 64, 900), (600, 160, 70000), (500, 128, 65601), (1400, 96, 900), (1300, 128, 900)]


def backward(h, W, target, seed=0, **more):
    z = h.double().nan_to_num(0, 0, 0) @ W.double().t().contiguous()
    live = (target >= 0) & (target < W.shape[0])
    lse = (torch.logsumexp(z, 1) * live).float()
    g = torch.randn(h.shape[0], generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    return gg.cross_entropy_backward(h, W, target, lse, g, **more), lse, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", WAYS)
def test_rows_without_a_target_may_hold_anything(T, D, V, dtype):
    """Their outputs are 0, and what they hold changes no bit of the others'."""
    say(f"masked rows T{T} D{D} V{V} {dtype}")
    h, W, target, _ = inputs(T, D, V, dtype, 0.4, T)
    dead = target < 0
    target[dead] = torch.randint(V, 1 << 30, (int(dead.sum()),), device="cuda").int()   # past the table, not only -100
    target[(dead.nonzero()[::2])[:, 0]] = -100
    bad = h.clone()
    bad[dead.nonzero()[:, 0][0::3]] = NAN
    bad[dead.nonzero()[:, 0][1::3]] = INF
    clean = torch.where(dead[:, None], torch.zeros_like(h), h)
    f0, f1 = gg.cross_entropy(clean, W, target), gg.cross_entropy(bad, W, target)
    assert torch.equal(f0["loss"], f1["loss"]) and torch.equal(f0["lse"], f1["lse"])
    assert not f1["loss"][dead].any() and not f1["lse"][dead].any()
    (b0, lse, g) = backward(clean, W, target)
    g = torch.where(dead, torch.full_like(g, NAN), g)                   # their gradient is not read either
    b1 = gg.cross_entropy_backward(bad, W, target, lse, g)
    assert torch.equal(b0["dh"], b1["dh"]) and torch.equal(b0["dW"], b1["dW"])
    assert not b1["dh"][dead].any() and bool(torch.isfinite(b1["dW"].float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", WAYS)
def test_no_row_takes_part(T, D, V, dtype):
    say(f"all masked T{T} D{D} V{V} {dtype}")
    h, W, target, _ = inputs(T, D, V, dtype, 1.0, T)
    f = gg.cross_entropy(h, W, target)
    assert not f["loss"].any() and not f["lse"].any()
    o = {"dh": torch.full_like(h, 7), "dW": torch.full_like(W, 7)}
    gg.cross_entropy_backward(h, W, target, f["lse"], torch.ones(T, device="cuda"), out=o)
    assert not o["dh"].any() and not o["dW"].any()
    ids, logits = torch.full((T, 3), -1, device="cuda", dtype=torch.int32), torch.zeros(T, 3, device="cuda")
    d = gg.distillation(h, W, ids, logits)
    assert not d["loss"].any() and not d["lse"].any() and not d["z"].any()
    b = gg.distillation_backward(h, W, ids, logits, d["z"], d["lse"], torch.ones(T, device="cuda"))
    assert not b["dh"].any() and not b["dW"].any()


@pytest.mark.parametrize("live", [1, 31, 32, 33, 255, 256, 257, 1279, 1280])
def test_listed_rows_end_at_every_border(live):
    """As many live rows as fit a block, a tile, a list, one more and one fewer, at the front, at the back and spread."""
    T, D, V = 1280, 128, 600
    say(f"{live} live rows of {T}")
    h, W, target, g = inputs(T, D, V, "bf16", 0.0, live)
    for where in ("front", "back", "spread"):
        order = torch.arange(T, device="cuda") if where == "front" else torch.arange(T - 1, -1, -1, device="cuda") if where == "back" else torch.randperm(T, device="cuda")
        t = torch.full_like(target, -1)
        t[order[:live]] = target[order[:live]]
        f = gg.cross_entropy(h, W, t)
        loss, far, lse, slack = loss64(h, W, t)
        within(f["loss"], loss, far, "loss")
        within(f["lse"], lse, slack, "lse")
        z, off = product(h, W, W.dtype)
        b = gg.cross_entropy_backward(h, W, t, f["lse"], g)
        hot = torch.zeros_like(z).scatter_(1, t.long().clamp(0, V - 1)[:, None], 1.0)
        (dh, x), (dW, y) = gradients64(h, W, z, off, lambda p: p - hot, 1.0, f["lse"], g, t >= 0, W.dtype)
        within(b["dh"], dh, x, "dh")
        within(b["dW"], dW, y, "dW")


@pytest.mark.parametrize("T,D,V", WAYS)
def test_a_row_that_is_no_number_keeps_it_to_itself(T, D, V):
    say(f"a NaN row T{T} D{D} V{V}")
    h, W, target, g = inputs(T, D, V, "bf16", 0.0, T + 1)
    f0 = gg.cross_entropy(h, W, target)
    bad = h.clone()
    bad[5, 3] = NAN
    f1 = gg.cross_entropy(bad, W, target)
    others = torch.arange(T, device="cuda") != 5
    assert math.isnan(float(f1["loss"][5])) and math.isnan(float(f1["lse"][5]))
    assert torch.equal(f0["loss"][others], f1["loss"][others])
    b0 = gg.cross_entropy_backward(h, W, target, f0["lse"], g, wanted=("dh",))
    b1 = gg.cross_entropy_backward(bad, W, target, f1["lse"], g, wanted=("dh",))
    assert b1["dW"] is None and bool(torch.isnan(b1["dh"][5].float()).all())
    assert torch.equal(b0["dh"][others], b1["dh"][others])


@pytest.mark.parametrize("T,D,V", [(7, 64, 300), (1100, 128, 300)])
def test_large_logits(T, D, V):
    """Logits from -3000 to 3000: the largest is taken off before an exponential."""
    h, W, target, _ = inputs(T, D, V, "bf16", 0.0, 3)
    h = (h.float() * 150).bfloat16()
    f = gg.cross_entropy(h, W, target)
    loss, far, lse, slack = loss64(h, W, target)
    assert float((h.float() @ W.float().t()).abs().max()) > 1000
    within(f["lse"], lse, slack, "lse")
    within(f["loss"], loss, far, "loss")


@pytest.mark.parametrize("tau", [0.25, 1.0])
@pytest.mark.parametrize("T", [20, 1200])
def test_teachers_with_masks_of_the_lowest_value(T, tau):
    """Entries at -infinity do not count, entries at the type's lowest value count with a probability of 0, unless all of a row are."""
    D, V, K = 64, 500, 6
    h, W, _, g = inputs(T, D, V, "f32", 0.0, 9)
    ids, logits = teacher(T, V, K, 4, masked=0.0)
    low = torch.finfo(torch.float32).min
    logits[0::4, 1:] = low
    logits[1::4] = low
    logits[2::4, 2:] = -INF
    logits[3::8] = -INF
    f = gg.distillation(h, W, ids, logits, temperature=tau)
    loss, far, lse, slack, z, zoff = distill64(h, W, ids, logits, tau)
    # a row's exponents of the lowest value are not roundings of anything: its bound without them
    far = torch.minimum(far, slack + 1e-5 * (loss.abs() + 10 + (z / tau).abs().amax(1)))
    within(f["loss"], loss, far, "loss")
    within(f["lse"], lse, slack, "lse")
    assert not f["loss"][3::8].any() and not f["lse"][3::8].any()
    b = gg.distillation_backward(h, W, ids, logits, f["z"], f["lse"], g, temperature=tau)
    assert bool(torch.isfinite(b["dh"]).all()) and not b["dh"][3::8].any()


def test_a_perfect_student_has_no_gradient():
    """A teacher whose K entries are the whole vocabulary, with the student's own logits: the loss and dz are roundings."""
    T, D, V = 50, 64, 200
    h, W, _, g = inputs(T, D, V, "f32", 0.0, 2)
    ids = torch.arange(V, device="cuda", dtype=torch.int32).expand(T, V).contiguous()
    logits = (h.double() @ W.double().t()).float()
    f = gg.distillation(h, W, ids, logits)
    b = gg.distillation_backward(h, W, ids, logits, f["z"], f["lse"], g)
    # each of z, logits, lse and q is off by at most (K + 100) u of a size of at most 60
    assert float(f["loss"].abs().max()) < 300 * U * 60 * 2
    assert float(b["dh"].abs().max()) < float(g.abs().max()) * 300 * U * 60 * 2 * float(W.abs().sum(0).max())


def test_the_same_entry_twice():
    """K entries that are all the same one are one entry of probability 1: cross entropy."""
    T, D, V, K = 300, 64, 900, 5
    h, W, target, g = inputs(T, D, V, "f32", 0.0, 6)
    ids, logits = target[:, None].expand(T, K).contiguous(), torch.randn(T, K, device="cuda")
    f, d = gg.cross_entropy(h, W, target), gg.distillation(h, W, ids, logits)
    q = torch.softmax(logits, 1)
    entropy = (q * q.log()).sum(1)
    assert float((d["loss"] - entropy - f["loss"]).abs().max()) < 1e-5
    a = gg.cross_entropy_backward(h, W, target, f["lse"], g)
    b = gg.distillation_backward(h, W, ids, logits, d["z"], d["lse"], g)
    for name in ("dh", "dW"):
        assert float((a[name] - b[name]).abs().max()) <= 1e-5 * float(a[name].abs().max())


@pytest.mark.parametrize("T,D,V,K", [(9, 64, 260, 4), (700, 64, 600, 4), (1200, 128, 600, 4)])
def test_gradients_against_differences(T, D, V, K):
    """The losses' own values, h and W moved both ways along a direction by 1e-2.  An fp32 loss of about 10 is off by less
    than 2e-5, a row's difference by 2e-3, rows independently: 6 standard deviations of their weighted sum.  The logits move by
    about 1e-2 with weights that sum to 1: the third order is below 1e-4 a row."""
    for name in ("loss", "distill"):
        h, W, target, g = inputs(T, D, V, "f32", 0.1, 11)
        ids, logits = teacher(T, V, K, 5)
        gen = torch.Generator(device="cuda").manual_seed(1)
        dh, dW = torch.randn(h.shape, generator=gen, device="cuda"), torch.randn(W.shape, generator=gen, device="cuda") * D ** -0.5

        def loss(h, W):
            return gg.cross_entropy(h, W, target) if name == "loss" else gg.distillation(h, W, ids, logits, temperature=2.0)

        f = loss(h, W)
        b = gg.cross_entropy_backward(h, W, target, f["lse"], g) if name == "loss" else \
            gg.distillation_backward(h, W, ids, logits, f["z"], f["lse"], g, temperature=2.0)
        step = 1e-2
        for what, a in (("dh", (dh, 0 * dW)), ("dW", (0 * dh, dW))):
            up, down = loss(h + step * a[0], W + step * a[1])["loss"], loss(h - step * a[0], W - step * a[1])["loss"]
            got = float((b[what].double() * (dh if what == "dh" else dW).double()).sum())
            want = float(((up.double() - down.double()) * g.double()).sum() / (2 * step))
            most = 6 * 2e-3 * float(g.double().square().sum().sqrt()) + 1e-4 * float(g.double().abs().sum())
            assert abs(got - want) <= most, (name, what, got, want, most)


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,D,V", WAYS + [(3, 33, 130), (1029, 31, 70), (255, 72, 300), (65, 72, 1100)])
def test_workspaces_and_outputs_of_just_their_size(T, D, V, dtype, grad):
    """A workspace of just the size, full of NaN, used twice; outputs between words that stay as they are."""
    say(f"sizes T{T} D{D} V{V} {dtype} {grad}")
    h, W, target, g = inputs(T, D, V, dtype, 0.2, 8)
    dt, gdt = TYPES[dtype], TYPES[grad]
    ids, logits = teacher(T, V, 9, 3)

    def between(shape, d):
        n = math.prod(shape)
        flat = torch.full((n + 256,), 3.0, dtype=d, device="cuda")
        return flat, flat[128:128 + n].view(shape)

    def guarded(f, out, need, names):
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        flats = {k: between(s, d) for k, (s, d) in out.items()}
        first = None
        for _ in range(2):
            r = f(out={k: v for k, (_, v) in flats.items()}, workspace=ws)
            got = {k: r[k].clone() for k in names}
            assert first is None or all(torch.equal(first[k], got[k]) for k in names)
            first = got
            for k, (flat, v) in flats.items():
                assert bool((flat[:128] == 3).all()) and bool((flat[128 + v.numel():] == 3).all()), k
        with pytest.raises(ValueError, match="needs"):
            f(out={}, workspace=ws[:-1])
        return first

    f32 = torch.float32
    a = guarded(lambda **k: gg.cross_entropy(h, W, target, **k), dict(loss=((T,), f32), lse=((T,), f32)),
                gg.cross_entropy_workspace_size(T, D, V, dt, False), ("loss", "lse"))
    plain = gg.cross_entropy(h, W, target)
    assert torch.equal(a["loss"], plain["loss"])
    b = guarded(lambda **k: gg.cross_entropy_backward(h, W, target, plain["lse"], g, grad_dtype=gdt, **k),
                dict(dh=((T, D), dt), dW=((V, D), gdt)), gg.cross_entropy_workspace_size(T, D, V, dt, True), ("dh", "dW"))
    c = gg.cross_entropy_backward(h, W, target, plain["lse"], g, grad_dtype=gdt)
    assert torch.equal(b["dh"], c["dh"]) and torch.equal(b["dW"], c["dW"])
    for one in ("dh", "dW"):
        o = gg.cross_entropy_backward(h, W, target, plain["lse"], g, grad_dtype=gdt, wanted=(one,))
        assert torch.equal(o[one], c[one]) and o["dW" if one == "dh" else "dh"] is None
    d = guarded(lambda **k: gg.distillation(h, W, ids, logits, **k), dict(loss=((T,), f32), lse=((T,), f32), z=((T, 9), f32)),
                gg.distillation_workspace_size(T, D, V, 9, dt, False), ("loss", "lse", "z"))
    guarded(lambda **k: gg.distillation_backward(h, W, ids, logits, d["z"], d["lse"], g, grad_dtype=gdt, **k),
            dict(dh=((T, D), dt), dW=((V, D), gdt)), gg.distillation_workspace_size(T, D, V, 9, dt, True), ("dh", "dW"))
    tokens = torch.where(target < 0, torch.full_like(target, V + 3), target)
    flat, y = between((T, D), dt)
    gg.embedding(tokens, W, out=y)
    assert bool((flat[:128] == 3).all()) and bool((flat[128 + y.numel():] == 3).all())
    need = gg.embedding_backward_workspace_size(T, D, V)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    flat, t = between((V, D), gdt)
    for _ in range(2):
        gg.embedding_backward(tokens, h, V, out=t, workspace=ws)
        assert bool((flat[:128] == 3).all()) and bool((flat[128 + t.numel():] == 3).all())
    assert torch.equal(t, gg.embedding_backward(tokens, h, V, grad_dtype=gdt))
    with pytest.raises(ValueError, match="needs"):
        gg.embedding_backward(tokens, h, V, workspace=ws[:-1])


def test_no_tokens():
    W = torch.randn(70, 24, device="cuda")
    h, none, f = W[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    assert gg.embedding(none, W).shape == (0, 24)
    assert not gg.embedding_backward(none, h, 70).any()
    out = W.clone()
    assert torch.equal(gg.embedding_backward(none, h, 70, out=out, accumulate=True), W)
    assert gg.cross_entropy(h, W, none)["loss"].shape == (0,)
    b = gg.cross_entropy_backward(h, W, none, f, f, out={"dW": out})
    assert not out.any() and b["dh"].shape == (0, 24)
    k = none.view(0, 1).expand(0, 5).contiguous()
    d = gg.distillation(h, W, k, torch.zeros(0, 5, device="cuda"))
    assert d["z"].shape == (0, 5)
    out = torch.full((70, 24), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.distillation_backward(h.bfloat16(), W.bfloat16(), k, d["z"], d["z"], f, f, out={"dW": out})
    assert not out.any()


@pytest.mark.parametrize("T,D,V", [(1, 64, 700), (300, 64, 2000), (1400, 128, 900)])
def test_captured_and_replayed(T, D, V):
    """Every call captured once into one graph and replayed with other inputs, eager calls in between on the same tensors."""
    say(f"captured T{T} D{D} V{V}")
    h, W, target, g = inputs(T, D, V, "bf16", 0.2, 1)
    ids, logits = teacher(T, V, 6, 2)
    shared = torch.zeros(V, D, device="cuda")

    def step():
        x = gg.embedding(target, W, scale=3.0)
        f = gg.cross_entropy(h, W, target)
        b = gg.cross_entropy_backward(h, W, target, f["lse"], g, out={"dW": shared})
        gg.embedding_backward(target, x, V, out=shared, accumulate=True)
        d = gg.distillation(h, W, ids, logits, temperature=2.0)
        e = gg.distillation_backward(h, W, ids, logits, d["z"], d["lse"], g, temperature=2.0)
        return [x, f["loss"], f["lse"], b["dh"], shared, d["loss"], d["z"], e["dh"], e["dW"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        h2, W2, t2, g2 = inputs(T, D, V, "bf16", 0.1 + 0.2 * k, 50 + k)
        i2, l2 = teacher(T, V, 6, 60 + k)
        for a, b in ((h, h2), (W, W2), (target, t2), (g, g2), (ids, i2), (logits, l2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (k, n)


def test_calls_on_two_streams_at_once():
    """Each stream's calls have workspaces of their own, and the current stream is neither."""
    sizes = [(1500, 128, 3000), (900, 64, 5000)]
    data = [inputs(*s, "bf16", 0.2, 20 + i) for i, s in enumerate(sizes)]

    def all_of(h, W, target, g, stream):
        f = gg.cross_entropy(h, W, target, stream=stream)
        b = gg.cross_entropy_backward(h, W, target, f["lse"], g, stream=stream)
        t = gg.embedding_backward(target, b["dh"], W.shape[0], stream=stream)
        return [f["loss"], b["dh"], b["dW"], t, gg.embedding(target, W, stream=stream)]

    want = [all_of(*d, None) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[] for _ in data]
        for k in range(4):
            for i, d in enumerate(data):
                got[i].append(all_of(*d, streams[i]))
        torch.cuda.synchronize()
        for i in range(2):
            for r in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_a_vocabulary_in_pieces():
    """dz of 2 GiB takes several pieces: dh is added up over them, dW written piece by piece."""
    T, D, V = 60000, 32, 50001
    say(f"pieces T{T} D{D} V{V}")
    h, W, target, g = inputs(T, D, V, "bf16", 0.1, 4)
    f = gg.cross_entropy(h, W, target)
    b = gg.cross_entropy_backward(h, W, target, f["lse"], g, grad_dtype=torch.float32)
    rows = torch.tensor([0, 1, 255, 256, 30000, 59998, 59999], device="cuda")
    loss, far, lse, slack = loss64(h[rows], W, target[rows])
    within(f["loss"][rows], loss, far, "loss")
    z, off = product(h[rows], W, W.dtype)
    live = target[rows] >= 0
    hot = torch.zeros_like(z).scatter_(1, target[rows].long().clamp(min=0)[:, None], 1.0)
    (dh, x), _ = gradients64(h[rows], W, z, off, lambda p: p - hot, 1.0, f["lse"][rows], g[rows], live, W.dtype)
    within(b["dh"][rows], dh, x, "dh")
    for v in (0, 17000, 17919, 17920, 35839, 35840, 50000):    # at and beside the pieces' borders, wherever they are
        w = W[v:v + 1]
        z, off = product(h, w, W.dtype)
        hot = (target == v).double()[:, None]
        # the softmax's denominator is that of all entries: in lse
        _, (dW, y) = gradients64(h, w, z, off, lambda p: p - hot, 1.0, f["lse"], g, target >= 0, torch.float32)
        within(b["dW"][v:v + 1], dW, y, f"dW {v}")


def test_offsets_past_32_bits():
    """A table of 2^31 elements and more: its last entries looked up, summed, and a loss's target."""
    D, V = 4096, 540000
    say(f"table of {V} x {D}")
    W = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 3, V - 1], dtype=torch.int32, device="cuda")
    W[ids.long()] = torch.randn(4, D, device="cuda").bfloat16()
    y = gg.embedding(ids, W)
    assert torch.equal(y, W[ids.long()])
    t = gg.embedding_backward(ids, y, V)
    assert torch.equal(t[V - 1], (2 * y[0].float()).bfloat16()) and torch.equal(t[V - 3], y[2]) and torch.equal(t[0], y[1])
    assert int((t != 0).any(1).sum()) == 3
    del t
    h = (torch.randn(4, D, device="cuda") * 0.05).bfloat16()
    f = gg.cross_entropy(h, W, ids)
    z = h.double() @ W[ids.long()[:3]].double().t()
    rest = torch.full((4, 1), math.log(V - 3), dtype=torch.float64, device="cuda")
    lse = torch.logsumexp(torch.cat([z, rest], 1), 1)
    at = torch.tensor([0, 1, 2, 0], device="cuda")
    assert float((f["lse"] - lse).abs().max()) < 1e-4
    assert float((f["loss"] - (lse - z.gather(1, at[:, None])[:, 0])).abs().max()) < 1e-4
    g = torch.ones(4, device="cuda")
    b = gg.cross_entropy_backward(h, W, ids, f["lse"], g)
    p = (z - lse[:, None]).exp()
    p[torch.arange(4), at] -= 1
    dh = p @ W[ids.long()[:3]].double()
    assert float((b["dh"].double() - dh).abs().max()) <= 2 ** -7 * float(dh.abs().max())
    dW = p.t().contiguous() @ h.double()
    got = b["dW"][ids.long()[:3]].double()
    assert float((got - dW).abs().max()) <= 2 ** -7 * float(dW.abs().max())


def test_rows_past_32_bits_of_dz():
    """dz of more than 2^32 bytes: few entries, many rows (one piece of 256 entries, rows of 512 bytes)."""
    T, D, V = 9_000_000, 8, 250
    say(f"rows {T}")
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    h = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    f = gg.cross_entropy(h, W, target)
    w = torch.full((T,), 1 / T, device="cuda")
    b = gg.cross_entropy_backward(h, W, target, f["lse"], w, grad_dtype=torch.float32)
    rows = torch.tensor([0, 4_194_304, 8_388_607, 8_388_608, T - 1], device="cuda")
    loss, far, lse, slack = loss64(h[rows], W, target[rows])
    within(f["loss"][rows], loss, far, "loss")
    z, off = product(h[rows], W, W.dtype)
    hot = torch.zeros_like(z).scatter_(1, target[rows].long()[:, None], 1.0)
    (dh, x), _ = gradients64(h[rows], W, z, off, lambda p: p - hot, 1.0, f["lse"][rows], w[rows], target[rows] >= 0, W.dtype)
    within(b["dh"][rows], dh, x, "dh")
    dW = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    mags = torch.zeros_like(dW)
    for t in range(0, T, 1_000_000):
        c = slice(t, t + 1_000_000)
        p = (h[c].double() @ W.double().t().contiguous() - f["lse"][c].double()[:, None]).exp()
        p[torch.arange(p.shape[0], device="cuda"), target[c].long()] -= 1
        p /= T
        dW += p.t().contiguous() @ h[c].double()
        mags += p.abs().t().contiguous() @ h[c].double().abs()
    # dz's half step of bf16 on every term, which random ones are far below; sums of 35000 terms at a time in fp32 and then of 256 parts
    within(b["dW"], dW, mags * (HALF[torch.bfloat16] + 40000 * U), "dW")
