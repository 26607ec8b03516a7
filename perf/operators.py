"""The operators of a training step that the benchmark measures: layer norm, the cross entropy of a
linear head, Newton-Schulz orthogonalisation and the Muon step, each with its cases, its plain form
and its definition in 64 bits."""
import math

import numpy as np
import torch

own = False

NS = (3.4445, -4.7750, 2.0315)  # the quintic's coefficients
NS_STEPS = 5
NS_EPS = 1e-7
LN_EPS = 1e-5
IGNORE = -100
MUON = {"lr": 3e-4, "momentum": 0.95, "weight_decay": 0.01}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Multiply-adds x 2 of the largest listed case: what a drawn case may cost at most.
MOST_FLOPS = 6 * 8192 * 4096 * 65536
# 64-bit products run at about 1 TFLOP/s: cases past this many flops have no exact().
MOST_EXACT = 1.6e13


def listed():
    return [
        # one token through the norm before a head: a call's latency
        {"name": "norm forward, one token", "op": "norm_forward", "rows": 1, "cols": 4096, "pad": 0,
         "dtype": "bf16", "beta": True},
        # a training batch of the Llama-sized decoder block
        {"name": "norm forward, batch", "op": "norm_forward", "rows": 16384, "cols": 4096, "pad": 0,
         "dtype": "bf16", "beta": True},
        # ragged fp32 widths (513) of the ragged unit, rows inside a wider buffer, a scale without offset
        {"name": "norm backward, ragged fp32", "op": "norm_backward", "rows": 1001, "cols": 513, "pad": 7,
         "dtype": "f32", "beta": False},
        {"name": "norm backward, batch", "op": "norm_backward", "rows": 16384, "cols": 4096, "pad": 0,
         "dtype": "bf16", "beta": True},
        # the loss of one token, without gradients (evaluation)
        {"name": "loss, one token", "op": "loss", "rows": 1, "cols": 512, "pad": 0, "vocab": 32000,
         "masked": 0.0, "grad": False},
        # a micro-batch of the 512-wide block's model
        {"name": "loss and gradients, micro-batch", "op": "loss", "rows": 256, "cols": 512, "pad": 0,
         "vocab": 32000, "masked": 0.0, "grad": True},
        # odd sizes everywhere, rows inside a wider buffer, a third of the targets ignored (prompts)
        {"name": "loss and gradients, ragged", "op": "loss", "rows": 1001, "cols": 513, "pad": 3,
         "vocab": 50021, "masked": 0.33, "grad": True},
        # a long batch of the 4096-wide model
        {"name": "loss and gradients, batch", "op": "loss", "rows": 8192, "cols": 4096, "pad": 0,
         "vocab": 65536, "masked": 0.0, "grad": True},
        # the ragged unit's odd matrices
        {"name": "orthogonalise, ragged", "op": "orthogonalise", "batch": 3, "rows": 1001, "cols": 513,
         "dtype": "f32"},
        # the four attention matrices of the 12 512-wide blocks at once
        {"name": "orthogonalise, 12 blocks", "op": "orthogonalise", "batch": 48, "rows": 512, "cols": 512,
         "dtype": "bf16"},
        # one 512-wide block's attention matrices on R = 4 ranks
        {"name": "muon, one block", "op": "muon", "batch": 4, "rows": 512, "cols": 512, "ranks": 4,
         "dtype": "bf16"},
        # W_gate of the Llama-sized block on R = 8 ranks
        {"name": "muon, W_gate", "op": "muon", "batch": 1, "rows": 14336, "cols": 4096, "ranks": 8,
         "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A size of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _flops(case):
    if case["op"] == "loss":
        return (6 if case["grad"] else 2) * case["rows"] * case["cols"] * case["vocab"]
    if case["op"] in ("orthogonalise", "muon"):
        k, n = sorted((case["rows"], case["cols"]))
        return case["batch"] * NS_STEPS * (2 * k * k * n * 2 + 2 * k * k * k)
    return 0


def draw(rng):
    while True:
        op = rng.choice(("norm_forward", "norm_backward", "loss", "loss", "orthogonalise", "muon"))
        case = {"op": op}
        if op.startswith("norm"):
            case |= {"rows": _spread(rng, 1, 32768), "cols": _spread(rng, 1, 16384), "pad": rng.choice((0, 0, 1, 8)),
                     "dtype": rng.choice(("bf16", "f32")), "beta": rng.random() < 0.5}
            fits = case["rows"] * case["cols"] <= 16384 * 4096
        elif op == "loss":
            case |= {"rows": _spread(rng, 1, 16384), "cols": _spread(rng, 8, 8192), "pad": rng.choice((0, 0, 1, 8)),
                     "vocab": _spread(rng, 100, 200000), "masked": rng.choice((0.0, 0.0, 0.1, 0.5, 0.9)),
                     "grad": rng.random() < 0.75}
            fits = case["rows"] * case["vocab"] <= 8192 * 65536 and case["cols"] * case["vocab"] <= 4096 * 131072
        elif op == "orthogonalise":
            case |= {"batch": _spread(rng, 1, 64), "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 1, 8192),
                     "dtype": rng.choice(("bf16", "f32"))}
            fits = case["batch"] * case["rows"] * case["cols"] <= 14336 * 4096
        else:
            case |= {"batch": _spread(rng, 1, 16), "rows": _spread(rng, 2, 14336), "cols": _spread(rng, 2, 14336),
                     "ranks": rng.choice((1, 2, 4, 8)), "dtype": rng.choice(("bf16", "f32"))}
            fits = case["batch"] * case["rows"] * case["cols"] <= 14336 * 4096
        if fits and _flops(case) <= MOST_FLOPS:
            return case


def _rows(gen, rows, cols, pad, dtype, scale=1.0, shift=0.0):
    """[rows, cols] values inside a buffer of cols + pad columns."""
    t = torch.empty(rows, cols + pad, device="cuda").normal_(0.0, scale, generator=gen)
    return (t + shift).to(dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda shape, scale: torch.empty(shape, device="cuda").normal_(0.0, scale, generator=gen)  # noqa: E731
    op = case["op"]
    s = {"op": op}
    if op.startswith("norm"):
        dt, n, d = DTYPES[case["dtype"]], case["rows"], case["cols"]
        s["x"] = _rows(gen, n, d, case["pad"], dt, 2.0, 0.3)
        s["gamma"] = (1.0 + normal((d,), 0.1)).to(dt)
        s["beta"] = normal((d,), 0.1).to(dt) if case["beta"] else None
        if op == "norm_backward":
            x = s["x"].float()
            s["dy"] = _rows(gen, n, d, case["pad"], dt, 1e-2)
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + LN_EPS)
    elif op == "loss":
        n, d, v = case["rows"], case["cols"], case["vocab"]
        s["hidden"] = _rows(gen, n, d, case["pad"], torch.bfloat16)
        s["weight"] = normal((v, d), 1.5 / math.sqrt(d)).to(torch.bfloat16)
        t = torch.randint(0, v, (n,), device="cuda", generator=gen)
        hide = torch.rand(n, device="cuda", generator=gen) < case["masked"]
        s["targets"] = torch.where(hide, torch.full_like(t, IGNORE), t)
        s["grad"] = case["grad"]
    elif op == "orthogonalise":
        s["g"] = normal((case["batch"], case["rows"], case["cols"]), 1e-3).to(DTYPES[case["dtype"]])
    else:
        b, m, n = case["batch"], case["rows"], case["cols"]
        s["master"] = list(normal((b, m, n), 1.0 / math.sqrt(n)).unbind(0))
        s["momentum"] = list(normal((b, m, n), 1e-3).unbind(0))
        s["params"] = [w.to(torch.bfloat16) for w in s["master"]]
        s["grads"] = [[normal((m, n), 1e-3).to(DTYPES[case["dtype"]]) for _ in range(case["ranks"])] for _ in range(b)]
    return s


# -- the plain forms ---------------------------------------------------------------

def _norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.square().mean(1) + LN_EPS)
    y = c * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_backward(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0).to(s["gamma"].dtype)}
    if s["beta"] is not None:
        out["dbeta"] = dy.sum(0).to(s["gamma"].dtype)
    return out


def _loss(s):
    h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"]
    valid = t != IGNORE
    count = valid.sum().clamp(min=1)
    at = torch.where(valid, t, torch.zeros_like(t))[:, None]
    logits = h @ w.t()
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    rows = (top + torch.log(total) - logits.gather(1, at))[:, 0]
    rows = torch.where(valid, rows, torch.zeros_like(rows))
    out = {"loss": rows.sum() / count, "row_loss": rows}
    if s["grad"]:
        scale = torch.where(valid, 1.0 / count, 0.0)[:, None]
        p = e / total
        p.scatter_add_(1, at, torch.full_like(total, -1.0))
        p = p * scale
        out["dhidden"] = (p @ w).to(torch.bfloat16)
        out["dweight"] = (p.t() @ h).to(torch.bfloat16)
    return out


def _newton_schulz(g):
    """[batch, m, n] in its own precision."""
    a, b, c = NS
    x = g / (g.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = g.shape[1] > g.shape[2]
    for _ in range(NS_STEPS):
        gram = x.transpose(1, 2) @ x if tall else x @ x.transpose(1, 2)
        poly = b * gram + c * (gram @ gram)
        x = a * x + (x @ poly if tall else poly @ x)
    return x


def _muon(s):
    """The R ranks' average gradient, momentum with Nesterov's look-ahead, the orthogonal update."""
    grads = torch.stack([torch.stack([q.float() for q in g]).sum(0) / len(g) for g in s["grads"]])
    mom = MUON["momentum"] * torch.stack(s["momentum"]) + grads
    u = _newton_schulz(grads + MUON["momentum"] * mom)
    scale = math.sqrt(max(1.0, u.shape[1] / u.shape[2]))
    w = torch.stack(s["master"]) * (1.0 - MUON["lr"] * MUON["weight_decay"]) - MUON["lr"] * scale * u
    torch._foreach_copy_(s["momentum"], list(mom))
    torch._foreach_copy_(s["master"], list(w))
    torch._foreach_copy_(s["params"], list(w.to(torch.bfloat16)))
    return {"master": s["master"], "momentum": s["momentum"], "params": s["params"]}


# -- the framework's operators -------------------------------------------------------

def _framework(s):
    import fully_sharded_state_gb300 as fsdp

    op = s["op"]
    if op == "norm_forward":
        y, mean, rstd = fsdp.layer_norm(s["x"], s["gamma"], s["beta"], eps=LN_EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dx, dgamma, dbeta = fsdp.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                                     with_beta=s["beta"] is not None)
        out = {"dx": dx, "dgamma": dgamma}
        return out if dbeta is None else out | {"dbeta": dbeta}
    if op == "loss":
        if not s["grad"]:
            loss, rows = fsdp.linear_cross_entropy(s["hidden"], s["weight"], s["targets"], ignore_index=IGNORE)
            return {"loss": loss, "row_loss": rows}
        loss, rows, dh, dw = fsdp.linear_cross_entropy_grad(s["hidden"], s["weight"], s["targets"],
                                                            ignore_index=IGNORE)
        return {"loss": loss, "row_loss": rows, "dhidden": dh, "dweight": dw}
    if op == "orthogonalise":
        return fsdp.newton_schulz(s["g"], steps=NS_STEPS, eps=NS_EPS, coefficients=NS)
    hp = fsdp.MuonHP(MUON["lr"], MUON["momentum"], MUON["weight_decay"])
    fsdp.muon_step(s["grads"], s["master"], s["momentum"], s["params"], hp)
    return {"master": s["master"], "momentum": s["momentum"], "params": s["params"]}


def run(state):
    if own:
        return _framework(state)
    op = state["op"]
    if op == "norm_forward":
        return _norm_forward(state)
    if op == "norm_backward":
        return _norm_backward(state)
    if op == "loss":
        return _loss(state)
    if op == "orthogonalise":
        return _newton_schulz(state["g"].float()).to(torch.bfloat16)
    return _muon(state)


# -- what a pass cannot do without -----------------------------------------------------

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        size = DTYPES[case["dtype"]].itemsize
        n, d = case["rows"], case["cols"]
        vectors = 2 if case["beta"] else 1
        if op == "norm_forward":
            return {"bytes": 2 * n * d * size + vectors * d * size + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * size + (1 + vectors) * d * size + 8 * n, "flops": 14 * n * d}
    if op == "loss":
        n, d, v = case["rows"], case["cols"], case["vocab"]
        kept = n * (1.0 - case["masked"])  # ignored rows need no product
        both = 2 if case["grad"] else 1
        return {"bytes": both * 2 * (n * d + v * d) + 12 * n,
                "flops": (6 if case["grad"] else 2) * kept * d * v}
    m, n, b = case["rows"], case["cols"], case["batch"]
    k, l = min(m, n), max(m, n)
    # the Gram product and its square are symmetric: half of each
    flops = b * NS_STEPS * (k * k * l + k * k * k + 2 * k * k * l)
    size = DTYPES[case["dtype"]].itemsize
    if op == "orthogonalise":
        return {"bytes": b * m * n * (size + 2), "flops": flops}
    return {"bytes": b * m * n * (case["ranks"] * size + 8 + 8 + 2), "flops": flops}


# -- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    if _flops(case) > MOST_EXACT:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        x = s["x"].double()
        n, d = x.shape
        gamma = s["gamma"].double()
        if op == "norm_forward":
            mu = x.sum(1) / d
            var = torch.einsum("ij,ij->i", x - mu[:, None], x - mu[:, None]) / d
            y = torch.einsum("ij,i,j->ij", x - mu[:, None], (var + LN_EPS).pow(-0.5), gamma)
            return {"y": y + (0 if s["beta"] is None else s["beta"].double()), "mean": mu, "rstd": (var + LN_EPS).pow(-0.5)}
        # the statistics are inputs of the backward pass
        z = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dy = s["dy"].double()
        dz = torch.einsum("ij,j->ij", dy, gamma)
        along = torch.einsum("ij,ij->i", dz, z) / d
        out = {"dx": (dz - dz.sum(1, keepdim=True) / d - along[:, None] * z) * s["rstd"].double()[:, None],
               "dgamma": torch.einsum("ij,ij->j", dy, z)}
        if case["beta"]:
            out["dbeta"] = dy.sum(0)
        return out
    if op == "loss":
        keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
        h, w = s["hidden"].double()[keep], s["weight"].double()
        t = s["targets"][keep]
        count = max(1, keep.numel())
        z = h @ w.t()
        lse = torch.logsumexp(z, 1)
        rows = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        rows[keep] = lse - z[torch.arange(keep.numel(), device="cuda"), t]
        out = {"loss": rows.sum() / count, "row_loss": rows}
        if case["grad"]:
            z = torch.exp_(z.sub_(lse[:, None]))
            z[torch.arange(keep.numel(), device="cuda"), t] -= 1.0
            z /= count
            dh = torch.zeros(case["rows"], case["cols"], dtype=torch.float64, device="cuda")
            dh[keep] = z @ w
            out |= {"dhidden": dh, "dweight": z.t() @ h}
        return out

    def orthogonal(g):
        """One matrix, by its wide side: p(X) = X (a + b S + c S^2), S = X^T X, of the transpose where that is smaller."""
        a, b, c = (np.float64(q) for q in NS)
        wide = g.shape[0] <= g.shape[1]
        x = g.t() if wide else g
        x = x / (torch.linalg.norm(x) + NS_EPS)
        eye = torch.eye(x.shape[1], dtype=torch.float64, device="cuda")
        for _ in range(NS_STEPS):
            gram = torch.mm(x.t(), x)
            x = torch.mm(x, torch.addmm(eye, gram, b * eye + c * gram, beta=a))
        return x.t() if wide else x

    if op == "orthogonalise":
        return torch.stack([orthogonal(g.double()) for g in s["g"]])
    out = {"master": [], "momentum": [], "params": []}
    for w, m, gs in zip(s["master"], s["momentum"], s["grads"]):
        g = sum(q.double() for q in gs) / len(gs)
        m = MUON["momentum"] * m.double() + g
        u = orthogonal(g + MUON["momentum"] * m) * max(1.0, case["rows"] / case["cols"]) ** 0.5
        w = w.double() * (1 - MUON["lr"] * MUON["weight_decay"]) - MUON["lr"] * u
        out["master"].append(w)
        out["momentum"].append(m)
        out["params"].append(w)
    return out
