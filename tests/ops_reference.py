"""Plain 64-bit forms of the training-step operators, for the tests."""
import torch

NS = (3.4445, -4.7750, 2.0315)
BF16_U = 2.0 ** -8   # unit roundoff of bf16: 8 significant bits
F16_U = 2.0 ** -11
F32_U = 2.0 ** -24


def layer_norm(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + eps).rsqrt()
    y = c * rstd[:, None] * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    dy, mean, rstd = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (x.double() - mean) * rstd
    g = dy * gamma.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0), xhat


def linear_cross_entropy(h, w, t, ignore, mean=True, scale=1.0):
    """row_loss, loss, dhidden, dweight and the sums of absolute terms that
    bound the rounding of G in the two gradients. Ignored rows are left out."""
    n = h.shape[0]
    keep = torch.nonzero((t != ignore) & (t >= 0) & (t < w.shape[0]))[:, 0]
    count = max(1, int((t != ignore).sum()))
    h64, w64 = h[keep].double(), w.double()
    z = h64 @ w64.t()
    lse = torch.logsumexp(z, 1)
    at = torch.arange(keep.numel(), device=h.device)
    rows = torch.zeros(n, dtype=torch.float64, device=h.device)
    rows[keep] = lse - z[at, t[keep]]
    bad = (t != ignore) & ((t < 0) | (t >= w.shape[0]))
    rows[bad] = float("nan")
    loss = rows.sum() / (count if mean else 1)
    g = torch.exp(z - lse[:, None])
    g[at, t[keep]] -= 1
    g *= scale / count if mean else scale
    put = lambda x: torch.zeros(n, h.shape[1], dtype=torch.float64, device=h.device).index_copy_(0, keep, x)  # noqa: E731
    return rows, loss, put(g @ w64), g.t() @ h64, put(g.abs() @ w64.abs()), g.abs().t() @ h64.abs()


def newton_schulz(g, steps=5, eps=1e-7, coef=NS):
    """One matrix."""
    a, b, c = coef
    x = g.double()
    x = x / (x.norm() + eps)
    tall = g.shape[0] > g.shape[1]
    for _ in range(steps):
        s = x.t() @ x if tall else x @ x.t()
        p = b * s + c * (s @ s)
        x = a * x + (x @ p if tall else p @ x)
    return x


def muon(grads, master, momentum, lr, mu, wd, scale, nesterov=True, **ns):
    """(master, momentum, size of the update) of one matrix."""
    g = sum(q.double() for q in grads) / len(grads)
    m = mu * momentum.double() + g
    u = newton_schulz(g + mu * m if nesterov else m, **ns) * (lr * scale)
    return master.double() * (1 - lr * wd) - u, m, u
