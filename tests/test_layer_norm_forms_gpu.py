"""Layer norm in the forms that many rows, and very wide ones, take: several
chunks a thread, a backward pass that fills its ring of stages again and again,
rows past the registers; and rows that start anywhere.

Tolerances as in test_layer_norm_gpu.py: a sum of n terms carries at most as
many units of 2^-24 of the sum of their absolute values as its longest chain of
additions is long. Forward: 32 values a thread and two trees, or for rows past
the registers cols / 1024 values a thread and 37 additions. The columns' sums:
a block's rows one after the other, then the blocks' (304 at most, 32 chains)."""
import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import layer_norm, layer_norm_backward

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, ref.BF16_U), "f32": (torch.float32, ref.F32_U)}
EPS = 1e-5
# rows that take every shape of the forward kernel where there are many, and
# more rows than 304 blocks have stages for in the backward kernel
SIZES = [(700, 1000), (20000, 512), (5000, 1024), (620, 1032), (7000, 2048), (3000, 4096), (700, 6000), (2600, 8192),
         (620, 12000), (1600, 16384), (613, 16392), (3, 30000), (2, 33000), (3, 32769), (4000, 264), (2500, 4088)]


def _make(rows, cols, dt, pad, first, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (r(rows, cols + pad) * 2 + 0.3).to(dt)[:, first:first + cols]
    dy = (r(rows, cols + pad) * 1e-2).to(dt)[:, first:first + cols]
    return x, dy, 1 + 0.1 * r(cols), 0.1 * r(cols)


def _within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} past the bound, worst {worst:.3g}x"


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,pdtype,pad,first,beta", [("bf16", "bf16", 0, 0, True), ("f32", "f32", 0, 0, False),
                                                         ("bf16", "f32", 8, 0, False), ("bf16", "bf16", 9, 1, True),
                                                         ("f32", "bf16", 5, 1, True)])
def test_layer_norm(cuda_lib, rows, cols, dtype, pdtype, pad, first, beta):
    """first: the rows begin that many elements into wider ones."""
    dt, u = DT[dtype]
    x, dy, gamma, off = _make(rows, cols, dt, pad, first, rows + cols)
    gamma, off = gamma.to(DT[pdtype][0]), off.to(DT[pdtype][0]) if beta else None
    chain = max(64, cols / 1024 + 37 + 8) * ref.F32_U
    y, mean, rstd = layer_norm(x, gamma, off, eps=EPS)
    wy, wm, wr = ref.layer_norm(x, gamma, off, EPS)
    size = x.double().abs() + wm.abs()[:, None]
    _within(mean, wm, chain * x.double().abs().mean(1), "mean")
    rel = chain + 4 * ref.F32_U * size.square().mean(1) * wr.square()
    _within(rstd, wr, rel * wr, "rstd")
    part = gamma.double().abs() * wr[:, None] * size
    _within(y, wy, u * wy.abs() + chain * part + rel[:, None] * wy.abs() + 4 * ref.F32_U * wy.abs(), "y")

    dx, dg, db = layer_norm_backward(dy, x, gamma, mean, rstd, with_beta=beta)
    wdx, wdg, wdb, xhat = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    g = (dy.double() * gamma.double()).abs()
    terms = g + g.mean(1, keepdim=True) + xhat.abs() * (g * xhat.abs()).mean(1, keepdim=True)
    xerr = 2 * ref.F32_U * size * rstd.double()[:, None]
    bound = u * wdx.abs() + chain * rstd.double()[:, None] * terms
    bound = bound + rstd.double()[:, None] * (xerr * (g * xhat.abs()).mean(1, keepdim=True) +
                                              xhat.abs() * (g * xerr).mean(1, keepdim=True))
    _within(dx, wdx, bound, "dx")
    up, long = DT[pdtype][1], (rows / 304 + 10 + 5 + 8 + 8) * ref.F32_U
    _within(dg, wdg, up * wdg.abs() + long * (dy.double() * xhat).abs().sum(0) + (dy.double().abs() * xerr).sum(0),
            "dgamma")
    if beta:
        _within(db, wdb, up * wdb.abs() + long * dy.double().abs().sum(0), "dbeta")
    for a, b in zip((y, mean, rstd, dx, dg), layer_norm(x, gamma, off, eps=EPS) +
                    layer_norm_backward(dy, x, gamma, mean, rstd, with_beta=beta)[:2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(40, 136), (900, 1024), (40, 4096), (900, 4096), (5, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_where_rows_start_changes_the_order_alone(cuda_lib, rows, cols, dtype):
    """The same values in rows that start on 16 bytes and in rows that do not:
    both within the bound of the exact statistics, though their sums may be
    formed in another order."""
    dt, u = DT[dtype]
    x, dy, gamma, beta = _make(rows, cols, dt, 0, 0, 9)
    wide = torch.zeros(rows, cols + 3, device="cuda", dtype=dt)
    wide[:, 1:1 + cols] = x
    moved = wide[:, 1:1 + cols]
    assert moved.data_ptr() % 16 != 0 and x.data_ptr() % 16 == 0
    one, two = layer_norm(x, gamma, beta), layer_norm(moved, gamma, beta)
    _, wm, wr = ref.layer_norm(x, gamma, beta, EPS)
    chain = max(64, cols / 1024 + 45) * ref.F32_U
    for _, mean, rstd in (one, two):
        _within(mean, wm, chain * x.double().abs().mean(1), "mean")
        size = (x.double().abs() + wm.abs()[:, None]).square().mean(1)
        _within(rstd, wr, (chain + 4 * ref.F32_U * size * wr.square()) * wr, "rstd")
    back = layer_norm_backward(dy, x, gamma, one[1], one[2]), layer_norm_backward(dy, moved, gamma, one[1], one[2])
    for a, b in zip(*back):
        assert ((a.double() - b.double()).abs() <= 2 * u * a.double().abs() + 2 * chain * a.double().abs().max()).all()
