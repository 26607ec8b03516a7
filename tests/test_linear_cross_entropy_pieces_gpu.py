"""Cross entropy of a linear head where 128-column pieces of the vocabulary
have no finite logit.

Tolerances as in test_linear_cross_entropy_gpu.py: z is off by at most
cols * 2^-23 * sum|h w| over the finite terms, the row loss by twice that and a
few fp32 units; G by its rounding to bf16, its fp16 exponential and z's error."""
import math

import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import linear_cross_entropy, linear_cross_entropy_grad

pytestmark = pytest.mark.gpu
IGNORE = -100


def _low(n, d, v, first, last, level):
    """Logits near `level` (times hidden 1), -inf for the words first..last."""
    g = torch.Generator(device="cuda").manual_seed(v + d)
    h = torch.randn(n, d, device="cuda", generator=g).bfloat16()
    w = (torch.randn(v, d, device="cuda", generator=g) / d ** 0.5).bfloat16()
    h[:, :2] = 1.0
    w[:, 0], w[:, 1] = 0.0, level
    w[first:last, 0] = float("-inf")
    words = torch.cat([torch.arange(first), torch.arange(last, v)]).cuda()
    t = words[torch.randint(0, len(words), (n,), device="cuda", generator=g)]
    return h, w, t, words


def _bounds(h, w, words, rows):
    fin = w[words].double()
    size = (h.double().abs() @ fin.abs().t()).max(1).values
    return 2 * (h.shape[1] * 2.0 ** -23 * size + 8 * ref.F32_U * (1 + rows.abs()))


@pytest.mark.parametrize("n,d,v,first,last", [(5, 64, 256, 0, 128), (50, 64, 700, 128, 640), (300, 128, 1500, 256, 1400),
                                              (64, 64, 384, 100, 300)])
@pytest.mark.parametrize("level", [-60.0, -100.0, -200.0, -2048.0])
def test_pieces_without_a_finite_logit(cuda_lib, n, d, v, first, last, level):
    """They count for nothing however low the others' logits are."""
    h, w, t, words = _low(n, d, v, first, last, level)
    wrows, wloss, wdh, wdw, adh, adw = ref.linear_cross_entropy(h, w, t, IGNORE)
    assert torch.isfinite(wrows).all() and torch.isfinite(wdw).all()
    err = _bounds(h, w, words, wrows)
    loss, rows = linear_cross_entropy(h, w, t)
    assert ((rows.double() - wrows).abs() <= err).all(), (rows.double() - wrows).abs().max()
    got = linear_cross_entropy_grad(h, w, t)
    assert torch.equal(got[0], loss) and torch.equal(got[1], rows)
    u = ref.BF16_U + ref.F16_U + 2 * err.max().item() + 16 * ref.F32_U
    tiny = 2.0 ** -24 / n
    # dhidden's column 0 is 0 * -inf, in the definition too
    bound = u * adh + ref.BF16_U * wdh.abs() + tiny * w[words].double().abs().sum(0)[None] + 1e-38
    assert torch.isnan(wdh[:, 0]).all() and torch.isnan(got[2][:, 0]).all()
    assert ((got[2].double() - wdh).abs() <= bound)[:, 1:].all()
    bound = u * adw + ref.BF16_U * wdw.abs() + tiny * h.double().abs().sum(0)[None] + 1e-38
    assert ((got[3].double() - wdw).abs() <= bound).all()
    gone = torch.ones(v, dtype=torch.bool, device="cuda")
    gone[words] = False
    assert not got[3][gone].any()


def test_one_column(cuda_lib):
    h = torch.ones(3, 1, device="cuda", dtype=torch.bfloat16)
    w = torch.full((256, 1), -100.0, device="cuda", dtype=torch.bfloat16)
    w[:128] = float("-inf")
    loss, rows = linear_cross_entropy(h, w, torch.tensor([128, 200, 255], device="cuda"))
    assert (rows - math.log(128)).abs().max() < 1e-5 and abs(loss.item() - math.log(128)) < 1e-5


def test_no_finite_logit_and_nan_pieces_stay_nan(cuda_lib):
    """A row of -inf alone has no softmax; a NaN among -inf is the row's."""
    h, w, t, words = _low(6, 64, 384, 128, 256, -200.0)
    w[130, 5] = float("nan")
    loss, rows, dh, dw = linear_cross_entropy_grad(h, w, t)
    assert torch.isnan(rows).all() and torch.isnan(loss) and torch.isnan(dw).all()
    h, w, t, words = _low(6, 64, 384, 128, 256, -200.0)
    w[:, 0] = float("-inf")
    loss, rows = linear_cross_entropy(h, w, t)
    assert torch.isnan(rows).all() and torch.isnan(loss)
