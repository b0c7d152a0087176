"""Embedding lookup, cross entropy and distillation over a large vocabulary, each with its gradient: cases, plain forms and exact values.

A case names its operator in "op":

  embed         y[t] = scale * table[ids[t]]; a row of zeros where ids[t] is not in [0, V)
  embed_grad    dtable[v] = scale * sum of dy[t] over the tokens with ids[t] = v (added to dtable where "add" is true)
  loss          z = h W^T;  lse[t] = log sum_v exp z[t, v];  loss[t] = lse[t] - z[t, target[t]]; both 0 where target[t] is not in [0, V)
  loss_grad     dz[t, v] = g[t] (exp(z[t, v] - lse[t]) - [v = target[t]]);  dh = dz W, dW = dz^T h
  distill       q[t] = softmax of the teacher's K logits / tau over the row's ids in [0, V);  lse[t] = log sum_v exp(z[t, v] / tau)
                loss[t] = sum_k q[t, k] (log q[t, k] - z[t, ids[t, k]] / tau) + lse[t]; z at the ids too, for the gradient
  distill_grad  dz[t, v] = g[t] / tau (exp(z[t, v] / tau - lse[t]) - sum of q[t, k] over ids[t, k] = v);  dh = dz W, dW = dz^T h

Sizes: rows are tokens (one in decoding, 512 in a small chunk, 4096 to 32768 in training), D the layer's width, V the entries of
the vocabulary, each a row of the table [V, D] that both ends of a model may share.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decoding step
        {"name": "embed_1x768", "op": "embed", "T": 1, "D": 768, "V": 50001, "dtype": "bf16"},
        # the training step's tokens
        {"name": "embed_32768x768", "op": "embed", "T": 32768, "D": 768, "V": 65536, "dtype": "bf16"},
        # a small chunk's gradient: writing the table's rows, nearly all zeros, is most of it
        {"name": "embed_grad_512x768", "op": "embed_grad", "T": 512, "D": 768, "V": 32768, "dtype": "bf16", "grad": "bf16", "add": False},
        # the training step's gradient, added to that of a table which the model's output shares
        {"name": "embed_grad_32768x768", "op": "embed_grad", "T": 32768, "D": 768, "V": 65536, "dtype": "bf16", "grad": "f32", "add": True},
        # the loss of one token: the whole table is read for it
        {"name": "loss_1x768", "op": "loss", "T": 1, "D": 768, "V": 50001, "dtype": "bf16", "masked": 0.0},
        # full precision, odd numbers of rows and entries
        {"name": "loss_4097x1000_f32", "op": "loss", "T": 4097, "D": 1000, "V": 20011, "dtype": "f32", "masked": 0.1},
        # the training step's tokens
        {"name": "loss_32768x768", "op": "loss", "T": 32768, "D": 768, "V": 65536, "dtype": "bf16", "masked": 0.0},
        # a small chunk's gradient
        {"name": "loss_grad_512x768", "op": "loss_grad", "T": 512, "D": 768, "V": 32768, "dtype": "bf16", "masked": 0.0},
        # fine-tuning: the prompts' tokens have no target
        {"name": "loss_grad_16384x768", "op": "loss_grad", "T": 16384, "D": 768, "V": 50001, "dtype": "bf16", "masked": 0.25},
        # a teacher's 64 largest logits a token
        {"name": "distill_2049x1024", "op": "distill", "T": 2049, "D": 1024, "V": 32768, "K": 64, "tau": 1.0, "dtype": "bf16", "masked": 0.0},
        # full precision, a small vocabulary
        {"name": "distill_grad_1000x512_f32", "op": "distill_grad", "T": 1000, "D": 512, "V": 16001, "K": 16, "tau": 1.5, "dtype": "f32", "masked": 0.1},
        # a student's training step
        {"name": "distill_grad_8192x1024", "op": "distill_grad", "T": 8192, "D": 1024, "V": 65536, "K": 64, "tau": 2.0, "dtype": "bf16", "masked": 0.0},
    ]


def _spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "loss", "loss_grad", "distill", "distill_grad"))
    while True:
        case = {"op": op, "T": _spread(rng, 1, 32768), "D": 8 * _spread(rng, 8, 256), "V": _spread(rng, 1000, 131072),
                "dtype": rng.choice(("bf16", "f32"))}
        if op == "embed":
            return case
        if op == "embed_grad":
            case["grad"] = rng.choice(("f32", case["dtype"]))
            case["add"] = rng.random() < 0.5
            return case
        case["masked"] = rng.choice((0.0, 0.0, 0.05, 0.4))
        if op in ("distill", "distill_grad"):
            case["K"] = _spread(rng, 1, 128)
            case["tau"] = rng.choice((1.0, 1.0, 2.0, 4.0))
        products = (1 if op in ("loss", "distill") else 3) * (3 if case["dtype"] == "f32" else 1)
        if products * case["T"] * case["V"] * case["D"] <= 3 * 16384 * 50001 * 768:
            return case


def _often(u, V):
    """Entries as a text has them, the first ones most often: about 1 / (v + 1)."""
    return (torch.exp(u * math.log(V + 1.0)).floor().long() - 1).clamp(0, V - 1).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op, T, D, V, dt = case["op"], case["T"], case["D"], case["V"], TYPES[case["dtype"]]
    s = dict(case)
    if op in ("embed", "embed_grad"):
        s["ids"] = _often(uniform(T), V)
        s["scale"] = math.sqrt(D)
        if op == "embed":
            s["table"] = (normal(V, D) / math.sqrt(D)).to(dt)
        else:
            s["dy"] = normal(T, D).to(dt)
            s["dtable"] = normal(V, D).to(TYPES[case["grad"]]) if case["add"] else None
        return s
    s["W"] = (normal(V, D) / math.sqrt(D)).to(dt)
    target = _often(uniform(T), V)
    # the rows behind the last norm, leaning towards what comes next: its probability lies between about 0.01 and 0.9
    lean = math.log(V) - 4.0 + 7.0 * uniform(T)
    s["h"] = (normal(T, D) + lean[:, None] * s["W"][target.long()].float()).to(dt)
    keep = uniform(T) >= case["masked"]
    s["g"] = uniform(T) / T
    if op in ("loss", "loss_grad"):
        s["target"] = torch.where(keep, target, torch.full_like(target, -100))
    else:
        # K entries of each row, all different: the next one among them, the others from anywhere
        K = case["K"]
        step = 1 + (uniform(T) * (V // (K + 1) - 1)).long().clamp(min=0)
        ids = (target.long()[:, None] + step[:, None] * torch.arange(K, device="cuda")) % V
        s["logits"] = normal(T, K) * 2.0
        s["logits"][:, 0] += 4.0
        # some rows have fewer than K
        ends = (uniform(T) < 0.1).float() * uniform(T) * K
        ids = torch.where(torch.arange(K, device="cuda") < K - ends[:, None], ids, torch.full_like(ids, -1))
        s["ids"] = torch.where(keep[:, None], ids, torch.full_like(ids, -1)).int()
    if op in ("loss_grad", "distill_grad"):  # what the forward pass left
        rows = max(1, (1 << 28) // V)
        W = s["W"].float().t()
        tau = case.get("tau", 1.0)
        z = [s["h"][t:t + rows].float() @ W / tau for t in range(0, T, rows)]
        lse = torch.cat([torch.logsumexp(p, 1) for p in z])
        if op == "loss_grad":
            s["lse"] = torch.where(keep, lse, torch.zeros_like(lse))
        else:
            s["lse"] = torch.where((s["ids"] >= 0).any(1), lse, torch.zeros_like(lse))
            at = s["ids"].long().clamp(min=0)
            parts = [p.gather(1, at[i * rows:i * rows + rows]) for i, p in enumerate(z)]
            s["z"] = torch.where(s["ids"] >= 0, torch.cat(parts) * tau, torch.zeros_like(s["logits"]))
    return s


def _embed(s):
    inside = (s["ids"] >= 0) & (s["ids"] < s["V"])
    y = s["table"][torch.where(inside, s["ids"], torch.zeros_like(s["ids"])).long()].float() * s["scale"]
    return (y * inside[:, None]).to(s["table"].dtype)


def _embed_grad(s):
    inside = (s["ids"] >= 0) & (s["ids"] < s["V"])
    dt = TYPES[s["grad"]]
    sums = torch.zeros(s["V"], s["D"], device=s["dy"].device)
    sums.index_add_(0, torch.where(inside, s["ids"], torch.zeros_like(s["ids"])).long(), s["dy"].float() * inside[:, None])
    sums = sums * s["scale"]
    if s["dtable"] is None:
        return sums.to(dt)
    s["dtable"].copy_(s["dtable"].float() + sums)
    return s["dtable"]


def _lse(z):
    top = z.max(1).values
    return top + torch.log(torch.exp(z - top[:, None]).sum(1))


def _loss(s):
    z = s["h"].float() @ s["W"].float().t()
    inside = (s["target"] >= 0) & (s["target"] < s["V"])
    at = torch.where(inside, s["target"], torch.zeros_like(s["target"])).long()
    lse = _lse(z)
    zero = torch.zeros_like(lse)
    return {"loss": torch.where(inside, lse - z.gather(1, at[:, None])[:, 0], zero), "lse": torch.where(inside, lse, zero)}


def _products(s, dz):
    dt = s["h"].dtype
    return {"dh": (dz @ s["W"].float()).to(dt), "dW": (dz.t() @ s["h"].float()).to(dt)}


def _loss_grad(s):
    z = s["h"].float() @ s["W"].float().t()
    inside = (s["target"] >= 0) & (s["target"] < s["V"])
    at = torch.where(inside, s["target"], torch.zeros_like(s["target"])).long()
    dz = torch.exp(z - s["lse"][:, None])
    dz.scatter_add_(1, at[:, None], -torch.ones_like(s["lse"])[:, None])
    return _products(s, torch.where(inside[:, None], dz * s["g"][:, None], torch.zeros_like(dz)))


def _teacher(s):
    """(entries that count, their ids or 0, q, log q)."""
    inside = (s["ids"] >= 0) & (s["ids"] < s["V"])
    at = torch.where(inside, s["ids"], torch.zeros_like(s["ids"])).long()
    a = torch.where(inside, s["logits"] / s["tau"], torch.full_like(s["logits"], -math.inf))
    a = a - a.max(1, keepdim=True).values.clamp(min=-3e38)
    e = torch.exp(a)
    total = e.sum(1, keepdim=True)
    q = torch.where(total > 0, e / total, torch.zeros_like(e))
    return inside, at, q, torch.where(q > 0, a - torch.log(total), torch.zeros_like(a))


def _distill(s):
    z = s["h"].float() @ s["W"].float().t()
    inside, at, q, logq = _teacher(s)
    some = inside.any(1)
    zk = torch.where(inside, z.gather(1, at), torch.zeros_like(q))
    lse = _lse(z / s["tau"])
    zero = torch.zeros_like(lse)
    loss = (q * (logq - zk / s["tau"])).sum(1) + lse
    return {"loss": torch.where(some, loss, zero), "lse": torch.where(some, lse, zero), "z": zk}


def _distill_grad(s):
    z = s["h"].float() @ s["W"].float().t()
    inside, at, q, _ = _teacher(s)
    dz = torch.exp(z / s["tau"] - s["lse"][:, None])
    dz.scatter_add_(1, at, -q)
    return _products(s, torch.where(inside.any(1)[:, None], dz * (s["g"] / s["tau"])[:, None], torch.zeros_like(dz)))


def run(state):
    s = state
    if own:
        import grouped_gemm_permute_amd as gg

        if s["op"] == "embed":
            return gg.embedding(s["ids"], s["table"], scale=s["scale"])
        if s["op"] == "embed_grad":
            if s["dtable"] is None:
                return gg.embedding_backward(s["ids"], s["dy"], s["V"], scale=s["scale"], grad_dtype=TYPES[s["grad"]])
            return gg.embedding_backward(s["ids"], s["dy"], s["V"], scale=s["scale"], out=s["dtable"], accumulate=True)
        if s["op"] == "loss":
            return gg.cross_entropy(s["h"], s["W"], s["target"])
        if s["op"] == "loss_grad":
            return gg.cross_entropy_backward(s["h"], s["W"], s["target"], s["lse"], s["g"])
        if s["op"] == "distill":
            return gg.distillation(s["h"], s["W"], s["ids"], s["logits"], temperature=s["tau"])
        return gg.distillation_backward(s["h"], s["W"], s["ids"], s["logits"], s["z"], s["lse"], s["g"], temperature=s["tau"])
    plain = {"embed": _embed, "embed_grad": _embed_grad, "loss": _loss, "loss_grad": _loss_grad, "distill": _distill,
             "distill_grad": _distill_grad}
    return plain[s["op"]](s)


def work(case):
    T, D, V, op = case["T"], case["D"], case["V"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "embed":
        return {"bytes": T * (4 + 2 * D * e), "flops": T * D}
    if op == "embed_grad":
        o = 2 if case["grad"] == "bf16" else 4
        rows = 2 * min(T, V) if case["add"] else V  # at the most, those that are read and written again
        return {"bytes": T * (4 + D * e) + rows * D * o, "flops": T * D}
    rows = T * (1.0 - case["masked"])
    entries = T * case["K"] * 12 if op == "distill" else T * case["K"] * 12 + 8 * T if op == "distill_grad" else 12 * T
    if op in ("loss", "distill"):
        return {"bytes": (T + V) * D * e + entries + 8 * T, "flops": 2 * rows * V * D}
    return {"bytes": 2 * (T + V) * D * e + entries, "flops": 6 * rows * V * D}


def _exact_teacher(s):
    """(entries that count, q, log q) row by row as weights over the largest."""
    inside = (s["ids"] >= 0) & (s["ids"] < s["V"])
    a = (s["logits"].double() / s["tau"]).masked_fill(~inside, -math.inf)
    some = inside.any(1, keepdim=True)
    logq = torch.where(some, a - torch.logsumexp(torch.where(some, a, torch.zeros_like(a)), 1, keepdim=True), torch.zeros_like(a))
    q = logq.exp().masked_fill(~inside, 0.0)
    return inside, q, logq.masked_fill(~inside, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op, T, D, V = case["op"], case["T"], case["D"], case["V"]
    if op == "embed":
        rows = s["ids"].long()
        return torch.index_select(s["table"].double(), 0, rows) * s["scale"]
    if op == "embed_grad":
        # tokens in the order of their entries; an entry's sum is the difference of two running sums
        order = torch.argsort(s["ids"].long(), stable=True)
        run_ = torch.cat([torch.zeros(1, D, dtype=torch.float64, device="cuda"), s["dy"].double()[order].cumsum(0)])
        ends = torch.searchsorted(s["ids"].long()[order], torch.arange(V + 1, device="cuda"))
        sums = (run_[ends[1:]] - run_[ends[:-1]]) * s["scale"]
        return sums if s["dtable"] is None else s["dtable"].double() + sums
    W, tau = s["W"].double(), case.get("tau", 1.0)
    Wt = W.t().contiguous()
    rows = max(1, (1 << 27) // V)
    out = {}
    if op in ("distill", "distill_grad"):
        inside, q, logq = _exact_teacher(s)
        at = s["ids"].long().clamp(min=0)
        live = inside.any(1)
    else:
        at = s["target"].long().clamp(min=0)
        live = s["target"] >= 0
    dW = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    parts = {"loss": [], "lse": [], "z": [], "dh": []}
    for t in range(0, T, rows):
        c = slice(t, t + rows)
        h = s["h"][c].double()
        z = torch.matmul(h, Wt)
        if op in ("loss", "distill"):
            lse = torch.logsumexp(z / tau, 1) * live[c]
            parts["lse"].append(lse)
            if op == "loss":
                parts["loss"].append((lse - z[torch.arange(z.shape[0], device="cuda"), at[c]]) * live[c])
            else:
                zk = torch.gather(z, 1, at[c]) * inside[c]
                parts["z"].append(zk)
                parts["loss"].append((lse + (q[c] * logq[c]).sum(1) - (q[c] * zk).sum(1) / tau) * live[c])
        else:
            p = z.div_(tau).sub_(s["lse"][c].double()[:, None]).exp_()
            if op == "loss_grad":
                p[torch.arange(p.shape[0], device="cuda"), at[c]] -= 1.0
            else:
                p.scatter_add_(1, at[c], -q[c])
            p *= (s["g"][c].double() / tau * live[c])[:, None]
            parts["dh"].append(torch.matmul(p, W))
            dW += torch.matmul(p.t().contiguous(), h)
    for name in {"loss": ("loss", "lse"), "distill": ("loss", "lse", "z")}.get(op, ("dh",)):
        out[name] = torch.cat(parts[name])
    if op in ("loss_grad", "distill_grad"):
        out["dW"] = dW
    return out
