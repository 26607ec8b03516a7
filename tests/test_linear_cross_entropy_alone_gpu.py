"""The loss without gradients, a batch of rows in pieces. Tolerance as in
test_linear_cross_entropy_gpu.py: the row losses are off by at most twice
cols * 2^-23 * sum|h w| and a few fp32 units."""
import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import linear_cross_entropy, linear_cross_entropy_grad

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.mark.parametrize("n,d,v,piece", [(300, 264, 1000, 64), (257, 96, 500, 256), (130, 40, 333, 1), (1000, 1032, 777, 320)])
@pytest.mark.parametrize("masked", [0.0, 0.6, 1.0])
def test_pieces(cuda_lib, n, d, v, piece, masked):
    g = torch.Generator(device="cuda").manual_seed(n)
    h = torch.randn(n, d, device="cuda", generator=g).bfloat16()
    w = (torch.randn(v, d, device="cuda", generator=g) * 1.5 / d ** 0.5).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    t[torch.rand(n, device="cuda", generator=g) < masked] = IGNORE
    loss, rows = linear_cross_entropy(h, w, t, piece_rows=piece)
    wrows, wloss = ref.linear_cross_entropy(h, w, t, IGNORE)[:2]
    size = (h.double().abs() @ w.double().abs().t()).max(1).values
    err = 2 * (d * 2.0 ** -23 * size + 8 * ref.F32_U * (1 + wrows.abs()))
    assert ((rows.double() - wrows).abs() <= err).all()
    assert (rows[t == IGNORE] == 0).all()
    count = max(1, int((t != IGNORE).sum()))
    assert abs(loss.item() - wloss.item()) <= (err.sum() + 32 * ref.F32_U * wrows.abs().sum()).item() / count
    # each row is its own piece's, with gradients or without
    got = linear_cross_entropy_grad(h, w, t, piece_rows=piece)
    assert torch.equal(got[0], loss) and torch.equal(got[1], rows)
    total, same = linear_cross_entropy(h, w, t, reduction="sum", piece_rows=piece)
    assert torch.equal(same, rows)
    assert abs(total.item() - wrows.sum().item()) <= (err.sum() + 32 * ref.F32_U * wrows.abs().sum()).item()
