"""The experts' products keep their sums in 32 bits in every form, sums in parts
and their join among them: shown by errors in the mean, which the worst case of K
roundings, a bound of each result, says little about.

A tensor core adds 16 products at a time to a sum and cuts it to 24 bits: K / 16
cuts that lean one way, less than 2^-23 of the sum's next power of two each, and K of
products that lean either way, which add up as their root: (K / 16 + sqrt(K)) 2^-22
of the sum's size.

Random terms. That, over all results, is what their root mean square may be off by
more than the 64-bit results rounded to bf16: a tenth for the longest K here, 9000.
Parts kept in 16 bits would make it the root of 2 of that or more.

Terms that cancel. Products c and -c in places of K far apart, among random ones of
size 1: the sums are near c in between, so results are off by their own rounding,
2^-8 of them at most, and (K / 16 + sqrt(K)) 2^-22 c in the mean: 0.16 for c = 1024
and K = 9000. A part of c in 16 bits is off by 2 in the mean."""
import pytest
import torch

import tuning_reference as tune
from fully_sharded_state_gb300 import grouped_linear, grouped_linear_backward, ops_wait_timeouts

pytestmark = pytest.mark.gpu

# rows, experts, n, k: sums in parts of each product, one kernel for both, tiles of one CTA and of two
SHAPES = [(300, 3, 40, 9000), (1, 2, 13, 4369), (20, 2, 9000, 104), (9000, 2, 130, 72), (5332, 1, 24, 16), (7001, 3, 96, 200),
          (1200, 6, 264, 136), (3000, 8, 256, 2048), (4000, 3, 2048, 512), (700, 5, 77, 513)]


@pytest.fixture(autouse=True)
def no_wait_given_up(cuda_lib):
    yield
    assert ops_wait_timeouts() == 0


def _make(rows, experts, n, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    cuts = torch.randint(0, rows + 1, (experts - 1,), device="cuda", generator=gen).sort().values
    return r(rows, k), r(rows, n), r(experts, n, k), torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows)])


def _all(x, dy, w, offsets):
    """(y, dx, dw), each with its 64-bit form."""
    o = offsets.tolist()
    wants = (tune.grouped_linear(x, w, o), *tune.grouped_linear_backward(dy, x, w, o))
    gots = (grouped_linear(x, w, offsets), *grouped_linear_backward(dy, x, w, offsets))
    return [(got, want) for got, (want, _) in zip(gots, wants)]


@pytest.mark.parametrize("rows,experts,n,k", SHAPES)
def test_random_terms(rows, experts, n, k):
    for (got, want), terms in zip(_all(*_make(rows, experts, n, k, rows + k)), (k, n, rows)):
        rms = lambda t: t.double().square().mean().sqrt()  # noqa: E731
        rounding = rms(want.float().bfloat16().double() - want)
        assert rms(got.double() - want) <= rounding + (terms / 16 + terms ** 0.5) * 2.0 ** -22 * rms(want)


@pytest.mark.parametrize("rows,experts,n,k", SHAPES)
def test_terms_that_cancel(rows, experts, n, k):
    x, dy, w, offsets = _make(rows, experts, n, k, rows + n)
    c = 1024.0
    # along k, along n, along an expert's rows: two places far apart whose products are c and -c
    if k >= 256:
        x[:, 3], x[:, k - 2] = c, -c
        w[:, :, 3] = w[:, :, k - 2] = 1.0
        got, want = grouped_linear(x, w, offsets), tune.grouped_linear(x, w, offsets.tolist())[0]
        _held(got, want, k, c)
    x, dy, w, offsets = _make(rows, experts, n, k, rows + n)
    if n >= 256:
        dy[:, 3], dy[:, n - 2] = c, -c
        w[:, 3] = w[:, n - 2] = 1.0
        got, want = grouped_linear_backward(dy, x, w, offsets)[0], tune.grouped_linear(dy, w.transpose(1, 2), offsets.tolist())[0]
        _held(got, want, n, c)
    x, dy, w, offsets = _make(rows, experts, n, k, rows + n)
    bounds = tune.bounds(offsets.tolist(), rows)
    long = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi - lo >= 256]
    for _, lo, hi in long:
        dy[lo + 3], dy[hi - 2] = c, -c
        x[lo + 3] = x[hi - 2] = 1.0
    dw = grouped_linear_backward(dy, x, w, offsets)[1]
    for e, lo, hi in long:
        _held(dw[e], dy[lo:hi].double().t() @ x[lo:hi].double(), hi - lo, c)


def _held(got, want, terms, c):
    err = (got.double() - want).abs().mean()
    assert err <= 2.0 ** -8 * want.abs().mean() + (terms / 16 + terms ** 0.5) * 2.0 ** -22 * c
