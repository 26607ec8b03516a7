"""The loss of a linear head and its gradients in every form that their products
have. On the host (no GPU) the shapes are held to reach them all; on a GPU each
is compared with the 64-bit form.

Tolerances as in test_linear_cross_entropy_gpu.py: z is off by at most
cols * 2^-23 * sum|h w|, G by its rounding to bf16, its fp16 exponential and
z's error; the gradients sum that and are rounded to bf16 themselves. With the
rows in pieces dweight is a sum of fp32 sums, whose rounding is below that."""
import pytest
import torch

import ops_plan
import ops_reference as ref

IGNORE = -100
# (rows, cols, vocabulary, elements between rows, piece_rows, share of rows ignored)
CASES = [
    (3, 33, 20522, 0, 0, 0.0), (3, 1801, 19512, 0, 0, 0.0), (3, 1800, 19512, 0, 0, 0.0), (200, 1100, 300, 0, 0, 0.1),
    (180, 5351, 40, 0, 0, 0.0), (180, 5352, 40, 0, 0, 0.0), (5, 65, 40, 0, 0, 0.0), (5, 72, 40, 0, 0, 0.0),
    (300, 31, 200, 0, 0, 0.2), (300, 32, 200, 0, 0, 0.2), (3, 31, 200, 0, 0, 0.0), (166, 33, 600, 0, 0, 0.0),
    (166, 40, 600, 0, 0, 0.0), (700, 180, 30011, 0, 0, 0.3), (3, 207, 5938, 0, 0, 0.0), (3, 208, 5938, 0, 0, 0.0),
    (3, 2345, 1833, 0, 0, 0.0), (3, 2344, 1833, 0, 0, 0.0), (1001, 513, 3001, 7, 0, 0.33), (1001, 511, 3001, 1, 0, 0.33),
    (130, 208, 5938, 0, 64, 0.2), (130, 2344, 1833, 0, 64, 0.0), (130, 65, 40, 7, 64, 0.0), (600, 264, 9000, 0, 256, 0.1),
    (300, 207, 5938, 0, 100, 0.2), (15, 40, 38, 0, 0, 0.0), (6, 35, 172, 0, 0, 0.0), (2654, 1787, 10, 0, 0, 0.1),
    (2602, 1744, 28, 0, 0, 0.0), (6, 8, 300, 0, 0, 0.0),
]


def _forms(n, d, v, pad, piece, masked):
    mapped = (d + pad) % 8 == 0
    out = set()
    for p in ops_plan.linear_cross_entropy(n, d, v, aligned=mapped, piece_rows=piece):
        if p["kind"] == "product":
            what = p["what"].split("(")[1].rstrip(")")
            if what == "logits":
                out.add((what, p["ctas"], p["tile"], int(p["parts"] > 0)))
            elif what == "dhidden":
                out.add((what, p["ctas"], p["tile"], int(p["splits"] > 1), int(d % 8 == 0)))
            else:
                out.add((what, p["ctas"], p["tile"], "sum" if 0 < piece < n else "rows" if d % 8 or not mapped else "map"))
    return out


def test_the_shapes_reach_every_form():
    got = set().union(*[_forms(*c) for c in CASES])
    want = {("logits", ctas, 256, long) for ctas in (1, 2) for long in (0, 1)}
    want |= {("dhidden", ctas, tile, 0, even) for ctas, tile in ((1, 64), (1, 128), (1, 256), (2, 256)) for even in (0, 1)}
    want |= {("dhidden", ctas, 256, 1, even) for ctas in (1, 2) for even in (0, 1)}
    want |= {("dweight", ctas, tile, how) for ctas, tile in ((1, 64), (1, 128), (1, 256), (2, 256))
             for how in ("rows", "map", "sum")}
    assert want <= got, sorted(want - got, key=str)


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,v,pad,piece,masked", CASES)
def test_loss_and_gradients(cuda_lib, n, d, v, pad, piece, masked):
    from fully_sharded_state_gb300 import linear_cross_entropy, linear_cross_entropy_grad

    g = torch.Generator(device="cuda").manual_seed(n + d + v)
    h = torch.randn(n, d + pad, device="cuda", generator=g).bfloat16()[:, :d]
    w = (torch.randn(v, d + pad, device="cuda", generator=g) * 1.5 / d ** 0.5).bfloat16()[:, :d]
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    t[torch.rand(n, device="cuda", generator=g) < masked] = IGNORE
    got = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE, piece_rows=piece)
    wrows, wloss, wdh, wdw, adh, adw = ref.linear_cross_entropy(h, w, t, IGNORE)
    keep = t != IGNORE
    count = max(1, int(keep.sum()))
    size = (h.double().abs() @ w.double().abs().t()).max(1).values
    err = torch.where(keep, 2 * (d * 2.0 ** -23 * size + 8 * ref.F32_U * (1 + wrows.abs())), 0.0)
    assert ((got[1].double() - wrows).abs() <= err).all()
    assert abs(got[0].item() - wloss.item()) <= (err.sum() + 32 * ref.F32_U * wrows.abs().sum()).item() / count
    u = ref.BF16_U + ref.F16_U + 2 * err.max().item() + 16 * ref.F32_U
    tiny = 2.0 ** -24 / count
    bound = u * adh + ref.BF16_U * wdh.abs() + tiny * w.double().abs().sum(0)[None] + 1e-38
    assert ((got[2].double() - wdh).abs() <= bound).all(), ((got[2].double() - wdh).abs() / bound).max()
    assert not got[2][~keep].any()
    hk = torch.where(keep[:, None], h.double().abs(), 0.0)
    bound = u * adw + ref.BF16_U * wdw.abs() + tiny * hk.sum(0)[None] + 1e-38
    assert ((got[3].double() - wdw).abs() <= bound).all(), ((got[3].double() - wdw).abs() / bound).max()
    loss, rows = linear_cross_entropy(h, w, t, ignore_index=IGNORE, piece_rows=piece)
    assert torch.equal(rows, got[1]) and torch.equal(loss, got[0])
    again = linear_cross_entropy_grad(h, w, t, ignore_index=IGNORE, piece_rows=piece)
    for a, b in zip(again, got):
        assert torch.equal(a, b)
