"""Layer norm (forward, backward), Newton-Schulz orthogonalisation and the Muon step: cases, plain forms and exact values.

A case names its operator in "op":

  norm       h = x (+ residual), y = (h - mean) rstd w + b   (rms: no mean); outputs y, h, mean, rstd
  norm_grad  the vector-Jacobian product of the same: dx (+ the gradient that reaches h by itself), dweight, dbias
  ortho      X = G / (|G| + eps); `steps` times X <- a X + (b A + c A A) X with A = X X^T on the shorter side
  muon       momentum <- beta momentum + dW; W <- (1 - lr wd) W - lr scale ortho(dW + beta momentum)

Sizes: rows are tokens in front of the layer (one in decoding, 512 in a small chunk, 4096 to 32768 in training), D its width;
matrices are the experts' weights, [E, D, F] or [E, F, D], and the router's [D, E].
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
LN_EPS = 1e-5
LR, BETA, DECAY = 0.02, 0.95, 0.01
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decoding step, in front of the router
        {"name": "norm_1x768", "op": "norm", "T": 1, "D": 768, "dtype": "bf16", "rms": False, "affine": True, "residual": True},
        # the training step's tokens: the residual sum and the norm in one pass
        {"name": "norm_32768x768", "op": "norm", "T": 32768, "D": 768, "dtype": "bf16", "rms": False, "affine": True, "residual": True},
        # full precision, an odd width and an odd number of rows
        {"name": "norm_4097x1001_f32", "op": "norm", "T": 4097, "D": 1001, "dtype": "f32", "rms": False, "affine": True, "residual": False},
        # a small chunk's backward, where launches count
        {"name": "norm_grad_512x768", "op": "norm_grad", "T": 512, "D": 768, "dtype": "bf16", "rms": False, "affine": True, "residual": False},
        # the training step's backward, with the residual stream's gradient added
        {"name": "norm_grad_32768x768", "op": "norm_grad", "T": 32768, "D": 768, "dtype": "bf16", "rms": False, "affine": True, "residual": True},
        # the wider layer in full precision, root mean square only
        {"name": "norm_grad_16384x1024_f32", "op": "norm_grad", "T": 16384, "D": 1024, "dtype": "f32", "rms": True, "affine": True, "residual": False},
        # the router's matrix
        {"name": "ortho_768x8", "op": "ortho", "B": 1, "M": 768, "N": 8, "dtype": "f32", "steps": 5},
        # one odd-sized matrix held in half the bits
        {"name": "ortho_1000x333_bf16", "op": "ortho", "B": 1, "M": 1000, "N": 333, "dtype": "bf16", "steps": 5},
        # the eight experts' up projections
        {"name": "ortho_8x768x1536", "op": "ortho", "B": 8, "M": 768, "N": 1536, "dtype": "f32", "steps": 5},
        # the shared expert's down projection, bf16 weights alone
        {"name": "muon_1536x768_bf16", "op": "muon", "B": 1, "M": 1536, "N": 768, "dtype": "bf16", "copy": False, "steps": 5},
        # the eight experts' down projections: 32-bit weights with the bf16 copy that the layer reads
        {"name": "muon_8x1536x768", "op": "muon", "B": 8, "M": 1536, "N": 768, "dtype": "f32", "copy": True, "steps": 5},
        # the sixteen experts of the wider layer
        {"name": "muon_16x1024x4096", "op": "muon", "B": 16, "M": 1024, "N": 4096, "dtype": "f32", "copy": False, "steps": 5},
    ]


def _spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _cost(case):
    m, n = min(case["M"], case["N"]), max(case["M"], case["N"])
    return case["B"] * case["steps"] * (4 * m * m * n + 2 * m**3)


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "ortho", "muon"))
    if op in ("norm", "norm_grad"):
        D = _spread(rng, 4, 8192)
        T = _spread(rng, 1, min(65536, 16384 * 1024 // D))
        return {"op": op, "T": T, "D": D, "dtype": rng.choice(("bf16", "f32")), "rms": rng.random() < 0.3,
                "affine": rng.random() < 0.8, "residual": rng.random() < 0.5}
    while True:
        case = {"op": op, "B": _spread(rng, 1, 16), "M": _spread(rng, 4, 4096), "N": _spread(rng, 4, 4096),
                "dtype": rng.choice(("bf16", "f32")), "steps": rng.randint(3, 6)}
        if op == "muon":
            case["copy"] = case["dtype"] == "f32" and rng.random() < 0.5
        if _cost(case) <= 16 * 5 * (4 * 1024 * 1024 * 4096 + 2 * 1024**3):
            return case


def _gradient(case, normal):
    """A weight's gradient as a batch of tokens leaves it: some strong directions over a floor of noise."""
    B, M, N = case["B"], case["M"], case["N"]
    r = max(1, min(M, N) // 16)
    return 1e-3 * (normal(B, M, r) @ normal(B, r, N) * (2.0 / math.sqrt(r)) + normal(B, M, N))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dt = TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        T, D = case["T"], case["D"]
        # the residual stream: unit noise, an offset for each feature, one feature in about 64 much larger
        large = 1.0 + 9.0 * (torch.rand(D, generator=g, device="cuda") < 1 / 64)
        s["x"] = (normal(T, D) * large + 0.5 * normal(D)).to(dt)
        s["r"] = (0.3 * normal(T, D)).to(dt) if case["residual"] else None
        s["w"] = (1.0 + 0.1 * normal(D)).to(dt) if case["affine"] else None
        s["b"] = (0.1 * normal(D)).to(dt) if case["affine"] else None
        if case["op"] == "norm_grad":
            s["dy"] = normal(T, D).to(dt)
            x = s["x"].double()
            mean = torch.zeros(T, dtype=torch.float64, device="cuda") if case["rms"] else x.mean(1)
            s["rstd"] = (1.0 / ((x - mean[:, None]).square().mean(1) + LN_EPS).sqrt()).float()
            s["mean"] = None if case["rms"] else mean.float()
    elif case["op"] == "ortho":
        s["G"] = _gradient(case, normal).to(dt)
    else:
        B, M, N = case["B"], case["M"], case["N"]
        s["W"] = (normal(B, M, N) / math.sqrt(M)).to(dt)
        s["dW"] = _gradient(case, normal)
        s["m"] = 10.0 * _gradient(case, normal)
        s["copy_out"] = s["W"].to(torch.bfloat16) if case["copy"] else None
    return s


def _scale(case):
    return math.sqrt(max(1.0, case["N"] / case["M"]))


def _norm(s):
    dt = TYPES[s["dtype"]]
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(dt)
    f = h.float()
    mean = None
    if not s["rms"]:
        mean = f.mean(1)
        f = f - mean[:, None]
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + LN_EPS)
    y = f * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"].float() + s["b"].float()
    return {"y": y.to(dt), "h": h, "mean": mean, "rstd": rstd}


def _norm_grad(s):
    dt = TYPES[s["dtype"]]
    dy = s["dy"].float()
    z = s["x"].float()
    if not s["rms"]:
        z = z - s["mean"][:, None]
    z = z * s["rstd"][:, None]
    g = dy if s["w"] is None else dy * s["w"].float()
    t = g - z * (g * z).mean(1, keepdim=True)
    if not s["rms"]:
        t = t - g.mean(1, keepdim=True)
    dx = t * s["rstd"][:, None]
    if s["r"] is not None:
        dx = dx + s["r"].float()
    out = {"dx": dx.to(dt), "dweight": None, "dbias": None}
    if s["w"] is not None:
        out["dweight"] = (dy * z).sum(0)
        out["dbias"] = dy.sum(0)
    return out


def _ortho(G, steps):
    a, b, c = COEFFS
    tall = G.shape[1] > G.shape[2]
    X = (G.transpose(1, 2) if tall else G).float().contiguous()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(steps):
        A = torch.matmul(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    return X.transpose(1, 2) if tall else X


def run(state):
    s = state
    if own:
        import grouped_gemm_permute_amd as gg

        if s["op"] == "norm":
            return gg.layer_norm(s["x"], s["w"], s["b"], residual=s["r"], eps=LN_EPS, rms=s["rms"])
        if s["op"] == "norm_grad":
            return gg.layer_norm_backward(s["x"], s["dy"], s["rstd"], mean=s["mean"], weight=s["w"], dh=s["r"],
                                          bias_grad=s["w"] is not None)
        if s["op"] == "ortho":
            return gg.newton_schulz(s["G"], steps=s["steps"], coeffs=COEFFS, eps=NS_EPS)
        gg.muon_step(s["W"], s["dW"], s["m"], LR, beta=BETA, weight_decay=DECAY, scale=_scale(s), steps=s["steps"],
                     coeffs=COEFFS, eps=NS_EPS, W_bf16=s["copy_out"])
        return {"W": s["W"], "momentum": s["m"], "copy": s["copy_out"]}
    if s["op"] == "norm":
        return _norm(s)
    if s["op"] == "norm_grad":
        return _norm_grad(s)
    if s["op"] == "ortho":
        return _ortho(s["G"], s["steps"]).to(TYPES[s["dtype"]]).contiguous()
    s["m"].mul_(BETA).add_(s["dW"])
    O = _ortho(s["dW"] + BETA * s["m"], s["steps"])
    W = (1.0 - LR * DECAY) * s["W"].float() - (LR * _scale(s)) * O
    s["W"].copy_(W)
    if s["copy_out"] is not None:
        s["copy_out"].copy_(W)
    return {"W": s["W"], "momentum": s["m"], "copy": s["copy_out"]}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        n = case["T"] * case["D"]
        if case["op"] == "norm":
            params = 2 * case["D"] * e if case["affine"] else 0
            return {"bytes": n * e * (4 if case["residual"] else 2) + params + 4 * case["T"] * (1 if case["rms"] else 2), "flops": 8 * n}
        params = case["D"] * (e + 8) if case["affine"] else 0
        return {"bytes": n * e * (4 if case["residual"] else 3) + params + 4 * case["T"] * (1 if case["rms"] else 2), "flops": 14 * n}
    size = case["B"] * case["M"] * case["N"]
    m, n, k = min(case["M"], case["N"]), max(case["M"], case["N"]), case["steps"]
    # the two symmetric products need one half of their entries; the iteration runs on X, or on X X^T alone with X multiplied once
    flops = case["B"] * min(k * (3 * m * m * n + m**3), 3 * m * m * n + (4 * k - 3) * m**3)
    if case["op"] == "ortho":
        return {"bytes": 2 * size * e, "flops": flops}
    return {"bytes": size * (12 + 2 * e + (2 if case["copy"] else 0)), "flops": flops}


def _exact_ortho(G, steps):
    """Every step multiplies X by a polynomial of A = X X^T, and those commute: the factors are gathered on the short side."""
    a, b, c = COEFFS
    G = G.double()
    if G.shape[1] > G.shape[2]:
        return _exact_ortho(G.transpose(1, 2), steps).transpose(1, 2)
    norm = torch.linalg.vector_norm(G, dim=(1, 2), keepdim=True) + NS_EPS
    A = torch.matmul(G, G.transpose(1, 2).contiguous()) / norm.square()
    I = torch.eye(A.shape[1], dtype=torch.float64, device=A.device)
    Q = I.expand_as(A).contiguous()
    for _ in range(steps):
        P = a * I + torch.matmul(A, b * I + c * A)
        Q = torch.matmul(Q, P)
        A = torch.matmul(P, torch.matmul(A, P))
    return torch.matmul(Q, G.contiguous()) / norm


def exact(case, seed):
    s = prepare(case, seed)
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(dt).double()  # h is stored, and the norm is the stored row's
        mean = h.sum(1) / case["D"]
        var = (h * h).sum(1) / case["D"] if case["rms"] else (h - mean[:, None]).pow(2).sum(1) / case["D"]
        rstd = (var + LN_EPS).rsqrt()
        y = (h if case["rms"] else h - mean[:, None]) * rstd[:, None]
        if s["w"] is not None:
            y = torch.addcmul(s["b"].double(), y, s["w"].double())
        return {"y": y, "h": h, "mean": None if case["rms"] else mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        rstd = s["rstd"].double()[:, None]
        z = s["x"].double() if case["rms"] else s["x"].double() - s["mean"].double()[:, None]
        dy = s["dy"].double()
        g = dy if s["w"] is None else dy * s["w"].double()
        # the Jacobian of a row: rstd (1 - [1 1^T / D] - z z^T rstd^2 / D)
        dx = rstd * g - rstd.pow(3) * z * (z * g).sum(1, keepdim=True) / case["D"]
        if not case["rms"]:
            dx = dx - rstd * g.sum(1, keepdim=True) / case["D"]
        if s["r"] is not None:
            dx = dx + s["r"].double()
        affine = s["w"] is not None
        return {"dx": dx, "dweight": (dy * z * rstd).sum(0) if affine else None, "dbias": dy.sum(0) if affine else None}
    if case["op"] == "ortho":
        return _exact_ortho(s["G"], case["steps"]).contiguous()
    m = BETA * s["m"].double() + s["dW"].double()
    O = _exact_ortho(s["dW"].double() + BETA * m, case["steps"])
    W = s["W"].double() - LR * (DECAY * s["W"].double() + _scale(case) * O)
    return {"W": W, "momentum": m, "copy": W.clone() if case["copy"] else None}
