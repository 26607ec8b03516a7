"""Layer norm, forward and backward, against its 64-bit form.

Tolerances. A result y is one rounding to its type (unit u: 2^-8 in bf16,
2^-24 in fp32) of a value formed in fp32. There, x - mean carries the error of
the mean and of one subtraction, each a few units of |x| + |mean|; sums over n
terms that go through trees of depth about 16 + log2(n) carry at most that
many units of the sum of their absolute terms: below 64 units at every size
here (fp32 chains of 16 per thread, then the tree, then the blocks)."""
import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import layer_norm, layer_norm_backward

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, ref.BF16_U), "f32": (torch.float32, ref.F32_U)}
CHAIN = 64 * ref.F32_U
EPS = 1e-5

SIZES = [(1, 1), (1, 4096), (3, 7), (5, 513), (2, 32), (9, 512), (17, 520), (33, 1000), (4, 1025), (70, 4096),
         (3, 8192), (2, 16384), (2, 16385), (3, 20000), (700, 96), (1300, 2048)]


def _make(rows, cols, dt, pad, seed, shift=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (r(rows, cols + pad) * 2 + shift).to(dt)[:, :cols]
    dy = (r(rows, cols + pad) * 1e-2).to(dt)[:, :cols]
    return x, dy, 1 + 0.1 * r(cols), 0.1 * r(cols)


def _within(got, want, bound, what):
    bad = (got.double() - want).abs() > bound
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} past the bound, worst {worst:.3g}x"


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,pdtype,pad,beta", [("bf16", "bf16", 0, True), ("bf16", "f32", 1, False),
                                                   ("f32", "f32", 0, False), ("f32", "bf16", 3, True),
                                                   ("bf16", "bf16", 8, True)])
def test_layer_norm(cuda_lib, rows, cols, dtype, pdtype, pad, beta):
    dt, u = DT[dtype]
    x, dy, gamma, off = _make(rows, cols, dt, pad, 7 * rows + cols)
    gamma, off = gamma.to(DT[pdtype][0]), off.to(DT[pdtype][0]) if beta else None
    y, mean, rstd = layer_norm(x, gamma, off, eps=EPS)
    wy, wm, wr = ref.layer_norm(x, gamma, off, EPS)
    size = x.double().abs() + wm.abs()[:, None]
    _within(mean, wm, CHAIN * x.double().abs().mean(1), "mean")
    # the variance's relative error: the mean's own squared, and the chain's
    rel = CHAIN + 4 * ref.F32_U * size.square().mean(1) * wr.square()
    _within(rstd, wr, rel * wr, "rstd")
    part = gamma.double().abs() * wr[:, None] * size
    _within(y, wy, u * wy.abs() + CHAIN * part + rel[:, None] * wy.abs() + 4 * ref.F32_U * wy.abs(), "y")

    dx, dg, db = layer_norm_backward(dy, x, gamma, mean, rstd, with_beta=beta)
    wdx, wdg, wdb, xhat = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    g = (dy.double() * gamma.double()).abs()
    terms = g + g.mean(1, keepdim=True) + xhat.abs() * (g * xhat.abs()).mean(1, keepdim=True)
    xerr = 2 * ref.F32_U * size * rstd.double()[:, None]  # of xhat, in the products
    bound = u * wdx.abs() + CHAIN * rstd.double()[:, None] * terms
    bound = bound + rstd.double()[:, None] * (xerr * (g * xhat.abs()).mean(1, keepdim=True) +
                                              xhat.abs() * (g * xerr).mean(1, keepdim=True))
    _within(dx, wdx, bound, "dx")
    up = DT[pdtype][1]
    _within(dg, wdg, up * wdg.abs() + 2 * CHAIN * (dy.double() * xhat).abs().sum(0) +
            (dy.double().abs() * xerr).sum(0), "dgamma")
    if beta:
        _within(db, wdb, up * wdb.abs() + 2 * CHAIN * dy.double().abs().sum(0), "dbeta")
    else:
        assert db is None


def test_no_rows_and_repeated_runs(cuda_lib):
    x, dy, gamma, beta = _make(0, 40, torch.float32, 0, 1)
    y, mean, rstd = layer_norm(x, gamma, beta)
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    dx, dg, db = layer_norm_backward(dy, x, gamma, mean, rstd)
    assert dx.shape == (0, 40) and not dg.any() and not db.any()
    x, dy, gamma, beta = _make(2000, 300, torch.bfloat16, 0, 2)
    first = None
    for _ in range(3):
        y, mean, rstd = layer_norm(x, gamma, beta)
        got = (y, mean, rstd) + layer_norm_backward(dy, x, gamma, mean, rstd)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_large_mean_keeps_the_variance(cuda_lib):
    # mean 1000, spread 2: sum(x^2) - mean^2 would lose it
    x, _, gamma, beta = _make(64, 1000, torch.float32, 0, 3, shift=1000.0)
    _, _, rstd = layer_norm(x, gamma, beta)
    want = ref.layer_norm(x, gamma, beta, EPS)[2]
    assert ((rstd.double() - want).abs() / want).max() < 1e-5


def test_infinities_and_nan_stay_in_their_row(cuda_lib):
    x, dy, gamma, beta = _make(6, 700, torch.float32, 0, 4)
    clean = layer_norm(x, gamma, beta)[0]
    x[1, 3], x[4, 699] = float("inf"), float("nan")
    y, mean, rstd = layer_norm(x, gamma, beta)
    others = [0, 2, 3, 5]
    assert torch.equal(y[others], clean[others])
    assert torch.isnan(y[4]).all() and torch.isnan(y[1, 3]) and not torch.isfinite(mean[1])


def test_outputs_given_as_views_and_another_stream(cuda_lib):
    """dgamma and dbeta as odd-offset views of one flat gradient buffer, out
    and dx inside wider buffers, on a stream of its own: nothing outside them
    changes."""
    rows, cols = 37, 130
    x, dy, gamma, beta = _make(rows, cols, torch.bfloat16, 5, 5)
    gamma, beta = gamma.bfloat16(), beta.bfloat16()
    want = layer_norm(x, gamma, beta)
    wantb = layer_norm_backward(dy, x, gamma, want[1], want[2])
    flat = torch.full((2 * cols + 7,), 9.0, device="cuda", dtype=torch.bfloat16)
    wide = torch.full((2, rows, cols + 9), 9.0, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = layer_norm(x, gamma, beta, out=wide[0, :, 3:3 + cols], stream=s)
    dx, dg, db = layer_norm_backward(dy, x, gamma, mean, rstd, dx=wide[1, :, 1:1 + cols], dgamma=flat[3:3 + cols],
                                     dbeta=flat[4 + cols:4 + 2 * cols], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip((y, mean, rstd, dx, dg, db), want + wantb):
        assert torch.equal(a, b)
    assert (flat[[0, 1, 2, 3 + cols, 2 * cols + 4, 2 * cols + 5, 2 * cols + 6]] == 9).all()
    assert (wide[0, :, :3] == 9).all() and (wide[0, :, 3 + cols:] == 9).all()
    assert (wide[1, :, :1] == 9).all() and (wide[1, :, 1 + cols:] == 9).all()


def test_gradients_against_differences(cuda_lib):
    """L = sum(y * r): central differences of the forward pass along random
    directions. Error: the step's third-order term (h^2 = 1e-4 of terms of
    order 1) and the differences' rounding, 2^-24 * sqrt(n) * |y r| / h."""
    rows, cols, h = 8, 200, 1e-2
    x, _, gamma, beta = _make(rows, cols, torch.float32, 0, 6)
    r = torch.randn(rows, cols, device="cuda")
    _, mean, rstd = layer_norm(x, gamma, beta)
    dx, dg, db = layer_norm_backward(r, x, gamma, mean, rstd)
    loss = lambda x, g, b: (layer_norm(x, g, b)[0].double() * r.double()).sum().item()  # noqa: E731
    for grad, at in ((dx, 0), (dg, 1), (db, 2)):
        args = [x, gamma, beta]
        d = torch.randn_like(args[at])
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * d, args[at] - h * d
        diff = (loss(*up) - loss(*down)) / (2 * h)
        want = (grad.double() * d.double()).sum().item()
        scale = (grad.double() * d.double()).norm().item()
        assert abs(diff - want) <= 2e-3 * scale + 1e-3, (at, diff, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(4, 1), (300, 1), (5, 64), (7, 513), (3, 2048), (2, 11127), (2, 20001)])
def test_rows_of_one_value(cuda_lib, rows, cols, dtype):
    """xhat is 0 in every element, and so dgamma, and with one column dx:
    differences of equal numbers, which are exact."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    value = (torch.randn(rows, 1, device="cuda", generator=g) * 2 + 0.3).to(dtype)
    x = value.expand(rows, cols).contiguous()
    dy = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    gamma = (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(dtype)
    mean, rstd = value.float()[:, 0].contiguous(), torch.full((rows,), 1e-5, device="cuda").rsqrt()
    dx, dgamma, dbeta = layer_norm_backward(dy, x, gamma, mean, rstd)
    assert not dgamma.any()
    if cols == 1:
        assert not dx.any()
    want = dy.double() * gamma.double()
    want = (want - want.mean(1, keepdim=True)) * rstd.double()[:, None]
    size = (dy.double() * gamma.double()).abs()
    # g rounded, its mean of up to 20,001 terms in a tree, one difference, one product, the result's rounding
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    bound = (64 * 2.0 ** -24 * (size + size.mean(1, keepdim=True))) * rstd.double()[:, None] + unit * want.abs() + 1e-30
    assert ((dx.double() - want).abs() <= bound).all()
