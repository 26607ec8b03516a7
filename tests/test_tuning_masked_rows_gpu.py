"""Rows that are masked or of no sequence count for nothing, whatever they hold, in
every form of the losses: one block, chunks of rows, many sequences over few rows."""
import pytest
import torch

from fully_sharded_state_gb300 import policy_loss, preference_loss

pytestmark = pytest.mark.gpu

# rows, sequences, rows before and behind them all
SIZES = [(700, 6, 33, 70), (8200, 2, 8, 0), (20000, 40, 300, 513), (20000, 2, 0, 9000), (70000, 500, 1, 31),
         (4000, 3000, 40, 100), (2500, 2100, 0, 0), (600000, 64, 1000, 77)]


def _make(rows, count, lead, tail):
    gen = torch.Generator(device="cuda").manual_seed(rows + count)
    cuts = torch.randint(0, rows - lead - tail + 1, (count - 1,), device="cuda", generator=gen).sort().values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows - lead - tail)]) + lead
    at = torch.arange(rows, device="cuda")
    mask = torch.rand(rows, device="cuda", generator=gen) < 0.6
    # the ends of what a warp has at once, and a whole sequence
    mask &= (at % 32 != 0) & (at % 256 != 255) & (at % 1024 < 1000)
    mask[offsets[count // 2]:offsets[count // 2 + 1]] = False
    counts = mask & (at >= lead) & (at < rows - tail)
    z = torch.empty(rows, device="cuda").exponential_(1.0, generator=gen)
    others = [(z + torch.randn(rows, device="cuda", generator=gen) * 0.2).abs() for _ in range(2)]
    fill = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda")[at % 4]
    spoilt = [torch.where(counts, t, fill.roll(i)) for i, t in enumerate((z, *others))]
    return (z, *others), spoilt, mask, counts, offsets, fill


def _same(got, want, weights, counts):
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(t.isfinite().all() for t in got)
    assert (weights[~counts] == 0).all() and (weights[counts] != 0).any()


@pytest.mark.parametrize("rows,count,lead,tail", SIZES)
@pytest.mark.parametrize("average", [False, True])
def test_preference(cuda_lib, rows, count, lead, tail, average):
    clean, spoilt, mask, counts, offsets, _ = _make(rows, count, lead, tail)
    loss = lambda z, old, ref: preference_loss(z, offsets, ref_row_loss=ref, mask=mask, average=average, beta=0.01)  # noqa: E731
    got = loss(*spoilt)
    _same(got, loss(*clean), got[2], counts)
    alone = lambda z: preference_loss(z, offsets, mask=mask, average=average, beta=0.01)  # noqa: E731
    got = alone(spoilt[0])
    _same(got, alone(clean[0]), got[2], counts)


@pytest.mark.parametrize("rows,count,lead,tail", SIZES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "sequence"])
def test_policy(cuda_lib, rows, count, lead, tail, reduction):
    clean, spoilt, mask, counts, offsets, fill = _make(rows, count, lead, tail)
    gen = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(rows, device="cuda", generator=gen)
    bad = torch.where(counts, a, fill)
    per = torch.randn(count, device="cuda", generator=gen)
    spoilt_per = per.clone()
    spoilt_per[count // 2] = float("nan")  # all of its rows are masked
    for x, y, by in ((a, bad, False), (per, spoilt_per, True)):
        loss = lambda z, old, ref, adv: policy_loss(z, old, adv, offsets=offsets, ref_row_loss=ref, mask=mask, kl_coef=0.1,  # noqa: E731
                                                    reduction=reduction, per_sequence=by)
        got = loss(*spoilt, y)
        _same(got, loss(*clean, x), got[1], counts)


@pytest.mark.parametrize("rows", [600, 20000])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_policy_without_sequences(cuda_lib, rows, reduction):
    clean, spoilt, mask, _, _, fill = _make(rows, 2, 0, 0)
    a = torch.randn(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    # what _make leaves out as a whole sequence holds finite numbers here, and counts
    mask = (torch.arange(rows, device="cuda") % 32 != 0) & (torch.arange(rows, device="cuda") % 5 != 3)
    spoilt = [torch.where(mask, t, fill) for t in clean]
    got = policy_loss(spoilt[0], spoilt[1], torch.where(mask, a, fill), ref_row_loss=spoilt[2], mask=mask, kl_coef=0.1,
                      reduction=reduction)
    want = policy_loss(clean[0], clean[1], a, ref_row_loss=clean[2], mask=mask, kl_coef=0.1, reduction=reduction)
    _same(got, want, got[1], mask)
