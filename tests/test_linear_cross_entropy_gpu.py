"""Cross entropy of a linear head against its 64-bit form.

Tolerances. z sums `cols` exact products in fp32: off by at most
cols * 2^-23 * sum|h w| (a chain of additions, each cut to 24 bits), so the
row loss, a log-sum-exp less one z, by twice that and a few fp32 units.
G is rounded once to bf16 (2^-8) after an fp16 exponential (2^-11, or 2^-25
of the tile's largest below fp16's normal range) with the error of z in the
exponent; the gradients sum G's error against |weight| and |hidden|, and are
rounded to bf16 themselves."""
import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import FsdpArgumentError, linear_cross_entropy, linear_cross_entropy_grad
from fully_sharded_state_gb300 import ops_wait_timeouts

pytestmark = pytest.mark.gpu
IGNORE = -100


def _make(n, d, v, seed, pad=0, masked=0.0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(n, d + pad, device="cuda", generator=g).bfloat16()[:, :d]
    w = (torch.randn(v, d + pad, device="cuda", generator=g) * scale / d ** 0.5).bfloat16()[:, :d]
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    t[torch.rand(n, device="cuda", generator=g) < masked] = IGNORE
    return h, w, t


def _check(h, w, t, got, mean=True, scale=1.0):
    loss, rows, dh, dw = got
    d = h.shape[1]
    wrows, wloss, wdh, wdw, adh, adw = ref.linear_cross_entropy(h, w, t, IGNORE, mean, scale)
    keep = t != IGNORE
    hz, wz = torch.nan_to_num(h.double().abs()), w.double().abs()
    dz = (d * 2 ** -23 * (hz @ wz.t()).max(1).values) + 8 * ref.F32_U * (1 + wrows.abs())
    err = torch.where(keep, 2 * dz, torch.zeros_like(dz))
    assert ((rows.double() - wrows).abs() <= err).all(), (rows.double() - wrows).abs().max()
    assert (rows[~keep] == 0).all()
    total = int(keep.sum())
    assert abs(loss.item() - wloss.item()) <= err.sum().item() / (max(1, total) if mean else 1) + \
        32 * ref.F32_U * wrows.abs().sum().item() / (max(1, total) if mean else 1)
    if dh is None:
        return
    s = scale / max(1, total) if mean else scale
    worst = err.max().item() if total else 0.0
    u = ref.BF16_U + ref.F16_U + 2 * worst + 16 * ref.F32_U
    tiny = 2.0 ** -24 * abs(s)
    bound = u * adh + ref.BF16_U * wdh.abs() + tiny * wz.sum(0)[None] + 1e-38
    assert ((dh.double() - wdh).abs() <= bound).all(), ((dh.double() - wdh).abs() / bound).max()
    assert (dh[~keep] == 0).all()
    hk = torch.where(keep[:, None], hz, torch.zeros_like(hz))
    bound = u * adw + ref.BF16_U * wdw.abs() + tiny * hk.sum(0)[None] + 1e-38
    assert ((dw.double() - wdw).abs() <= bound).all(), ((dw.double() - wdw).abs() / bound).max()


CASES = [(1, 8, 2, 0, 0.0), (1, 512, 1000, 0, 0.0), (2, 1, 1, 0, 0.0), (7, 33, 129, 1, 0.0), (64, 64, 256, 0, 0.0),
         (65, 100, 255, 0, 0.3), (128, 72, 257, 8, 0.0), (129, 200, 1000, 0, 0.5), (300, 513, 777, 3, 0.33),
         (1000, 264, 3001, 0, 0.1), (256, 512, 32000, 0, 0.0), (40, 1024, 5000, 0, 0.9), (700, 96, 20011, 0, 0.02)]


@pytest.mark.parametrize("n,d,v,pad,masked", CASES)
def test_loss_and_gradients(cuda_lib, n, d, v, pad, masked):
    h, w, t = _make(n, d, v, n + d + v, pad, masked)
    got = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    _check(h, w, t, got)
    loss, rows = linear_cross_entropy(h, w, t, ignore_index=IGNORE)
    assert torch.equal(loss, got[0]) and torch.equal(rows, got[1])
    assert ops_wait_timeouts() == 0


@pytest.mark.parametrize("n,d,v,piece", [(300, 264, 1000, 64), (257, 96, 500, 256), (130, 40, 333, 1), (512, 64, 4000, 128)])
@pytest.mark.parametrize("masked", [0.0, 0.6, 1.0])
def test_pieces_of_the_rows(cuda_lib, n, d, v, piece, masked):
    h, w, t = _make(n, d, v, 3 * n, 0, masked)
    _check(h, w, t, linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE, piece_rows=piece))


@pytest.mark.parametrize("n,d,v,pad", [(16, 1024, 100, 0), (16, 1025, 100, 0), (5, 2056, 300, 8), (16, 4100, 129, 0), (130, 8192, 40, 0)])
def test_long_rows(cuda_lib, n, d, v, pad):
    """Above 1024 columns the sums are of parts of 512. A part is 32 steps of
    16 products; each cuts the running sum, and the products aligned with it,
    to 24 bits: off by at most twice 2^-23 of the largest of them. Joining the
    parts rounds by 2^-24 of the running sum each."""
    h, w, t = _make(n, d, v, d, pad)
    got = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    _check(h, w, t, got)
    part = 512 if d > 1024 else d
    worst = torch.zeros(n, dtype=torch.float64, device="cuda")
    for r in range(n):
        z = h[r].double()[None] * w.double()  # [v, d]
        run, off = torch.zeros(v, dtype=torch.float64, device="cuda"), torch.zeros(v, dtype=torch.float64, device="cuda")
        for k in range(0, d, part):
            q = z[:, k:k + part].cumsum(1).abs()
            largest = torch.maximum(q.max(1).values, z[:, k:k + part].abs().max(1).values)
            off += -(-min(part, d - k) // 16) * 2.0 ** -22 * largest
            run += z[:, k:k + part].sum(1)
            off += 2.0 ** -24 * run.abs()
        worst[r] = off.max()
    wrows = ref.linear_cross_entropy(h, w, t, IGNORE, True, 1.0)[0]
    err = (got[1].double() - wrows).abs()
    # one z, and the log-sum-exp, a mean of them; 8 units for the logarithm,
    # the exponentials and the last sums
    assert (err <= 2 * worst + 8 * ref.F32_U * (1 + wrows.abs())).all(), (err / worst).max()
    loss, rows = linear_cross_entropy(h, w, t, ignore_index=IGNORE)
    assert torch.equal(loss, got[0]) and torch.equal(rows, got[1])
    assert ops_wait_timeouts() == 0


@pytest.mark.parametrize("scale", [1.0, 1024.0, -0.25])
def test_sum_and_scale(cuda_lib, scale):
    h, w, t = _make(150, 80, 600, 11, 0, 0.2)
    _check(h, w, t, linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE, reduction="sum", grad_scale=scale), False,
           scale)


def test_nothing_counts(cuda_lib):
    h, w, t = _make(70, 40, 300, 12)
    t.fill_(IGNORE)
    h.fill_(float("nan"))
    loss, rows, dh, dw = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    assert loss.item() == 0 and not rows.any() and not dh.any() and not dw.any()
    empty = h[:0]
    loss, rows, dh, dw = linear_cross_entropy_grad(empty, w, t[:0], ignore_index=IGNORE)
    assert loss.item() == 0 and rows.shape == (0,) and dh.shape == (0, 40) and not dw.any()


def test_ignored_rows_may_hold_anything(cuda_lib):
    h, w, t = _make(200, 96, 700, 13, 0, 0.4)
    want = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    gone = t == IGNORE
    h[gone] = float("nan")
    h[gone.nonzero()[0]] = float("inf")
    for a, b in zip(linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE), want):
        assert torch.equal(a, b)


def test_a_target_out_of_range_is_loud(cuda_lib):
    h, w, t = _make(20, 64, 300, 14)
    t[3], t[7] = 300, -1
    loss, rows, dh, dw = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    bad = torch.tensor([i in (3, 7) for i in range(20)], device="cuda")
    assert torch.isnan(loss) and torch.equal(torch.isnan(rows), bad)
    assert not dh[bad].any() and torch.isfinite(dw).all()


def test_large_logits_and_infinite_ones(cuda_lib):
    """Logits of some hundreds, and a vocabulary whose -inf logits fill whole
    tiles: their probability is 0, the others' as if they were not there."""
    h, w, t = _make(100, 64, 600, 15, scale=60.0)
    _check(h, w, t, linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE))
    h, w, t = _make(50, 64, 700, 16)
    h[:, 0] = 1.0
    t %= 128
    w[128:640, 0] = float("-inf")
    loss, rows = linear_cross_entropy(h, w, t)
    keep = torch.cat([torch.arange(128), torch.arange(640, 700)]).cuda()
    want = torch.logsumexp((h.double() @ w[keep].double().t()), 1) - (h.double() * w[t].double()).sum(1)
    assert ((rows.double() - want).abs() < 1e-4).all()


def test_nan_stays_in_its_row(cuda_lib):
    h, w, t = _make(60, 64, 500, 17)
    h[5, 1] = float("nan")
    loss, rows, dh, dw = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    bad = torch.arange(60, device="cuda") == 5
    assert torch.equal(torch.isnan(rows), bad) and torch.isnan(loss)
    assert torch.isnan(dh[5]).all() and torch.isfinite(dh[~bad]).all() and torch.isnan(dw).all()


def test_outputs_given_as_views_and_another_stream(cuda_lib):
    n, d, v = 90, 72, 400
    h, w, t = _make(n, d, v, 18, 0, 0.2)
    want = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    flat = torch.full((v * d + 11,), 9.0, device="cuda", dtype=torch.bfloat16)  # odd offset: a ragged unit's buffer
    wide = torch.full((n, d + 5), 9.0, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE, dweight=flat[5:5 + v * d].view(v, d),
                                    dhidden=wide[:, 2:2 + d], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (flat[:5] == 9).all() and (flat[5 + v * d:] == 9).all()
    assert (wide[:, :2] == 9).all() and (wide[:, 2 + d:] == 9).all()


def test_gradients_against_differences(cuda_lib):
    """Differences of the loss between two bf16 points, against the gradient at
    the point between them. Error: the third-order term, the rounding of the
    gradient (2^-7 of the terms) and of the losses (2^-22 of about 7)."""
    n, d, v = 24, 64, 300
    h, w, t = _make(n, d, v, 19)
    for which in (0, 1):
        base = (h, w)[which]
        step = (0.02 * torch.randn(base.shape, device="cuda")).bfloat16()
        up, down = (base + step), (base - step)
        mid = ((up.float() + down.float()) / 2).bfloat16()
        move = up.double() - down.double()
        args = lambda x: (x, w, t) if which == 0 else (h, x, t)  # noqa: E731
        diff = linear_cross_entropy(*args(up))[0].item() - linear_cross_entropy(*args(down))[0].item()
        grad = linear_cross_entropy_grad(*args(mid))[2 + which]
        want = (grad.double() * move).sum().item()
        scale = (grad.double() * move).norm().item()
        assert abs(diff - want) <= 0.05 * scale + 1e-5, (which, diff, want, scale)


def test_same_bits_every_time(cuda_lib):
    h, w, t = _make(333, 136, 5001, 20, 0, 0.3)
    first = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE)
    for _ in range(3):
        for a, b in zip(linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE), first):
            assert torch.equal(a, b)


def test_refusals(cuda_lib):
    h, w, t = _make(8, 16, 32, 21)
    for bad in (lambda: linear_cross_entropy(h.float(), w, t), lambda: linear_cross_entropy(h, w[:, :8], t),
                lambda: linear_cross_entropy(h, w, t.int()), lambda: linear_cross_entropy(h, w, t[:4]),
                lambda: linear_cross_entropy(h.t(), w, t), lambda: linear_cross_entropy(h, w.cpu(), t),
                lambda: linear_cross_entropy(h, w, t, reduction="none"),
                lambda: linear_cross_entropy_grad(h, w, t, dweight=torch.empty_like(w).float()),
                lambda: linear_cross_entropy_grad(h, w, t, dhidden=torch.empty_like(w))):
        with pytest.raises(FsdpArgumentError):
            bad()
    with pytest.raises(Exception, match="overlaps"):
        linear_cross_entropy_grad(h, w, t, dhidden=h)
