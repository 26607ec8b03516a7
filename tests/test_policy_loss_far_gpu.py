"""The policy loss where exp leaves fp32: rows whose log ratio or whose distance
from the reference model passes 88.7, or is infinite.

Tolerances, in units of 2^-24 (half a step): exp is good to 2 steps, of which a
far row takes two (8 units); the factors between them, the ratio's remainder and
the share of a row are a rounding each (6), and a lane's sum of 8 rows 8 more.
The distance from the reference model is rounded before its exponential is taken,
which is |d| units of that."""
import pytest
import torch

from ops_reference import F32_U
from fully_sharded_state_gb300 import policy_loss

pytestmark = pytest.mark.gpu

INF = float("inf")
ROWS = [64, 20000]  # one block; chunks


def _rand(rows, seed, lo=0.0, hi=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(rows, device="cuda", generator=gen) * (hi - lo) + lo


def _near(got, want, units):
    """Next to fp32's end, rounding decides whether it holds a number: either will do."""
    got, want = got.double().cpu(), want.cpu()
    ratio = want.abs() / torch.finfo(torch.float32).max
    over, held = ratio > 1.001, ratio < 0.999
    assert torch.equal(got[over], want[over].sign() * INF)
    err, bound = (got - want)[held].abs(), (units * F32_U * want.abs())[held]
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_ratios_that_overflow_with_a_remainder(cuda_lib, rows, sign):
    """old - now is not an fp32 number, and off it to either side."""
    now, old = _rand(rows, 1), _rand(rows, 2, 95.0, 140.0)
    rest = (old.double() - now.double()) - (old - now).double()
    assert (rest < 0).any() and (rest > 0).any()
    loss, weights, _, clipped = policy_loss(now, old, torch.full_like(now, sign))
    if sign < 0:
        # exp(95) / 20000 is 9e36, an fp32 number; most of the others are above
        want = -torch.exp(old.double() - now.double()).cpu() / rows
        _near(weights, want, 24)
        _near(loss, -want.sum(), 24)
        assert loss.item() == INF and clipped.item() == 0
    else:
        assert abs(loss.item() + 1.2) < 1e-5 and (weights == 0).all() and clipped.item() == 1


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("far", [99.5, INF])
def test_without_a_coefficient_the_reference_changes_neither_loss_nor_weights(cuda_lib, rows, far):
    now, old, ref = _rand(rows, 3, 0.0, 4.0), _rand(rows, 4, 0.0, 4.0), _rand(rows, 5, 0.0, 4.0)
    now[5::7] = far
    a = _rand(rows, 6, -1.0, 1.0)
    offsets = torch.tensor([0, rows // 3, rows], device="cuda")
    for reduction in ("mean", "sum", "sequence"):
        alone = policy_loss(now, old, a, offsets=offsets, reduction=reduction)
        watched = policy_loss(now, old, a, offsets=offsets, reduction=reduction, ref_row_loss=ref)
        assert alone[0].isfinite() and alone[1].isfinite().all()
        assert torch.equal(alone[0], watched[0]) and torch.equal(alone[1], watched[1])
        assert torch.equal(alone[3], watched[3]) and not watched[2].isfinite()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kl_coef", [0.0, 0.1])
@pytest.mark.parametrize("which", ["row_loss", "reference"])
def test_infinitely_far_from_the_reference(cuda_lib, rows, kl_coef, which):
    """exp(d) - 1 - d is infinite for d = inf, and for -inf; the other rows are as they were."""
    now, ref = _rand(rows, 3, 0.0, 4.0), _rand(rows, 5, 0.0, 4.0)
    old, a = now.clone(), torch.ones(rows, device="cuda")
    before = policy_loss(now, old, a, ref_row_loss=ref, kl_coef=kl_coef)
    (now if which == "row_loss" else ref)[7] = INF
    loss, weights, kl, _ = policy_loss(now, old, a, ref_row_loss=ref, kl_coef=kl_coef)
    assert kl.item() == INF
    others = torch.arange(rows, device="cuda") != 7
    assert torch.equal(weights[others], before[1][others])
    if kl_coef:
        assert loss.item() == INF
        # the ratio is 0 or 1, and exp(d) - 1 infinite or -1
        want = INF if which == "row_loss" else (1 - kl_coef) / rows
        assert weights[7].item() == pytest.approx(want, rel=1e-6)
    else:
        assert loss.isfinite()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("reduction", ["mean", "sum", "sequence"])
@pytest.mark.parametrize("to", [88.0, 96.0, 130.0])
def test_factors_that_bring_far_rows_back_into_range(cuda_lib, rows, reduction, to):
    """exp(l) A, kl_coef exp(d) and the mean of exp(d), with the share of a row, are
    fp32 numbers beyond where exp(l) and exp(d) are."""
    now, old = _rand(rows, 1), _rand(rows, 2, 60.0, to)
    now[::2], old[::2] = old[::2].clone(), now[::2].clone()  # every other row is far from the reference instead
    ref = now.clone()
    ref[::2] = old[::2]
    a = -10.0 ** _rand(rows, 3, -16.0, -1.0)
    a[::2] = 1.0
    kl_coef = 0.04
    offsets = torch.tensor([0, rows // 3, rows])
    got = policy_loss(now, old, a, offsets=offsets.cuda(), ref_row_loss=ref, kl_coef=kl_coef, reduction=reduction)
    z, o, r, c = (t.double().cpu() for t in (now, old, ref, a))
    n = torch.diff(offsets)
    share = {"mean": torch.ones(rows).double() / rows, "sum": torch.ones(rows).double(),
             "sequence": (0.5 / n.double()).repeat_interleave(n)}[reduction]
    ratio, d = torch.exp(o - z), z - r
    far = torch.expm1(d) - d
    term = kl_coef * far - torch.minimum(ratio * c, ratio.clamp(0.8, 1.2) * c)  # no far ratio's side is cut off
    _near(got[1], (ratio * c + kl_coef * torch.expm1(d)) * share, 24 + to)
    _near(got[0], (term * share).sum(), 24 + to)
    _near(got[2], far.mean(), 24 + to)
    assert got[3].item() == 0
