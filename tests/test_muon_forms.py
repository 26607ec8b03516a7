"""Newton-Schulz and the Muon step in every form that their kernels have.

The shapes below were chosen so that together they reach every form; on the
host (no GPU) they are held to it, so that a changed estimate cannot move them
elsewhere unseen. On a GPU every matrix of each is compared with the 64-bit
iteration.

Tolerances. Emulated on the CPU (fp16 operands, fp32 sums, x in 22 bits, the
shift), full-rank Gaussian matrices of 6 x 2886 to 1311 x 1428 come out 1.7e-3
to 2.1e-3 off in norm, bf16's rounding of the result included (1.7e-3), and at
most 4.2e-3 of the rms past that rounding in one element. Bounds: 4e-3 in norm
and 1.5e-2 of the rms per element beside the rounding (2^-8 of each). Below 16
rows or columns a matrix may have so few elements that their roundings do not
average out: 2^-8 + 1e-3 in norm there. For the Muon step, whose update is not
rounded, the first two of the update."""
import pytest
import torch

import ops_plan
import ops_reference as ref

# (matrices, m, n, ranks of a Muon step or 0)
CASES = [
    # the thin form; few matrices and many, x kept and x read twice
    (300, 2, 5, 0), (3, 30, 700, 0), (2, 400, 20, 0), (3, 8, 4000, 0), (3, 4000, 8, 0), (5, 2, 9, 2), (2, 40, 3, 3), (2, 20, 1500, 2),
    # a team of blocks: tiles of 64, 128 and 256 columns, of wide matrices and tall ones
    (1, 34, 37, 3), (1, 39, 34, 3), (1, 37, 40, 0), (1, 46, 35, 0), (4, 13, 2633, 0), (5, 14, 2199, 2),
    (40, 135, 67, 0), (39, 146, 72, 3), (12, 18, 1690, 0), (12, 21, 1650, 2), (42, 157, 146, 0), (39, 150, 140, 2),
    (4, 1000, 1000, 0),
    # teams that take a second matrix, and a third
    (248, 37, 34, 0), (239, 33, 42, 0), (247, 41, 124, 0), (269, 74, 71, 0), (135, 190, 133, 0), (127, 159, 189, 0),
    (400, 50, 60, 0),
    # a kernel per product: S in parts
    (8, 2606, 14, 0), (7, 2928, 12, 2), (6, 13, 2886, 0), (8, 14, 2493, 2), (20, 1810, 20, 2), (4, 137, 2820, 3),
    (2, 2996, 210, 2), (2, 132, 7500, 0), (1, 7600, 133, 3), (2, 140, 8000, 2), (3, 9000, 135, 0),
    # S whole, squares and their mirror images, rows that start on 16 bytes and rows that do not
    (105, 159, 85, 0), (53, 270, 67, 3), (51, 137, 304, 0), (378, 67, 78, 0), (40, 206, 257, 2), (51, 316, 149, 0),
    (2, 811, 1297, 2), (40, 429, 209, 0), (2, 1335, 805, 0), (1, 2792, 841, 0), (5, 1053, 908, 3), (1, 859, 2942, 0),
    (3, 1311, 1428, 3), (2, 2339, 853, 0), (2, 830, 2528, 0), (48, 512, 512, 0), (24, 512, 512, 2), (10, 1001, 513, 0),
    (16, 1024, 1024, 0), (2, 1536, 800, 2), (2, 800, 1536, 3), (3, 1424, 1312, 0),
]
# what the forms are told apart by; x: whether it is the next step's, the result or the master
TEAMS = {("team", tile, tall, muon, again) for tile in (64, 128, 256) for tall in (0, 1) for muon in (0, 1)
         for again in (0, 1) if not (muon and again)}  # 64 matrices at most: no second round
THIN = {("thin", tall, muon) for tall in (0, 1) for muon in (0, 1)}
PARTS = {("S, parts", ctas, tall) for ctas in (1, 2) for tall in (0, 1)} | {("S, sum",)}
SQUARES = {(what, ctas, tile, sym) for what in ("S", "P") for ctas, tile in ((1, 64), (1, 128), (2, 256)) for sym in (0, 1)}
SQUARES |= {("S", "tall", tall, sym) for tall in (0, 1) for sym in (0, 1)}
STEPS = {("x", ctas, tile, tall, then) for ctas, tile in ((1, 64), (1, 128), (1, 256), (2, 256)) for tall in (0, 1)
         for then in ("two units", "one unit", "result", "master")}
ROWS = {(then, vec) for then in ("result", "master") for vec in (0, 1)}


def _forms(batch, m, n, ranks):
    plan = ops_plan.newton_schulz(batch, m, n, ranks=ranks, steps=2)
    tall, muon, out = int(m > n), int(ranks > 0), set()
    for i, p in enumerate(plan):
        what = p["what"].split("(")[-1].rstrip(")")
        if p["kind"] == "team":
            out.add(("team", p["tile"], tall, muon, int(p["rounds"] > 1)))
        elif what == "thin":
            out.add(("thin", tall, muon))
        elif what == "S, parts":
            out.add((what, p["ctas"], tall))
        elif what == "S, sum":
            out.add((what,))
        elif what in ("S", "P"):
            out.add((what, p["ctas"], p["tile"], p["sym"]))
            if what == "S":
                out.add(("S", "tall", tall, p["sym"]))
        elif what == "x":
            then = ("master" if muon else "result") if i + 1 == len(plan) else "two units" if p["stages"] == 4 else "one unit"
            out.add(("x", p["ctas"], p["tile"], tall, then))
            if i + 1 == len(plan):
                out.add((then, int(n % 8 == 0)))
    return out


def test_the_shapes_reach_every_form():
    got = set().union(*[_forms(*c) for c in CASES])
    for want in (TEAMS, THIN, PARTS, SQUARES, STEPS, ROWS):
        assert want <= got, sorted(want - got, key=str)


def _exact(g, steps=5, eps=1e-7):
    """All matrices of [batch, m, n] at once, in 64 bits."""
    a, b, c = ref.NS
    x = g.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    if x.shape[1] > x.shape[2]:
        return _exact(g.transpose(1, 2), steps, eps).transpose(1, 2)
    for _ in range(steps):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x


def _gauss(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n", [c[:3] for c in CASES if not c[3]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_newton_schulz(cuda_lib, batch, m, n, dtype):
    from fully_sharded_state_gb300 import newton_schulz

    g = (_gauss(torch.Generator(device="cuda").manual_seed(m + n), batch, m, n) * 1e-3).to(dtype)
    out = newton_schulz(g)
    exact = _exact(g)
    off = out.double() - exact
    size = exact.square().sum((1, 2)).sqrt()
    norm = 4e-3 if min(m, n) >= 16 else ref.BF16_U + 1e-3
    assert (off.square().sum((1, 2)).sqrt() <= norm * size).all(), (off.square().sum((1, 2)).sqrt() / size).max()
    rms = size[:, None, None] / (m * n) ** 0.5
    assert (off.abs() <= ref.BF16_U * exact.abs() + 1.5e-2 * rms).all()
    assert torch.equal(newton_schulz(g), out)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n,ranks", [c for c in CASES if c[3]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_muon_step(cuda_lib, batch, m, n, ranks, dtype):
    """Momentum: the fold of the ranks and two fp32 operations per element."""
    from fully_sharded_state_gb300 import MuonHP, muon_step

    gen = torch.Generator(device="cuda").manual_seed(m + n)
    grads = [[(_gauss(gen, m, n) * 1e-3).to(dtype) for _ in range(ranks)] for _ in range(batch)]
    master, mom = [_gauss(gen, m, n) / n ** 0.5 for _ in range(batch)], [_gauss(gen, m, n) * 1e-3 for _ in range(batch)]
    params = [torch.zeros(m, n, device="cuda", dtype=torch.bfloat16) for _ in range(batch)]
    w0, m0 = torch.stack(master).double(), torch.stack(mom).double()
    lr, mu, wd = 0.02, 0.9, 0.1
    muon_step(grads, master, mom, params, MuonHP(lr=lr, momentum=mu, weight_decay=wd))
    folded = torch.stack([sum(q.double() for q in g) / ranks for g in grads])
    moved = mu * m0 + folded
    size = torch.stack([sum(q.double().abs() for q in g) / ranks for g in grads]) + m0.abs()
    assert ((torch.stack(mom).double() - moved).abs() <= (ranks + 4) * 2 * ref.F32_U * size).all()
    u = _exact(folded + mu * moved) * (lr * max(1.0, m / n) ** 0.5)
    want = w0 * (1 - lr * wd) - u
    off = torch.stack(master).double() - want
    near = 4 * ref.F32_U * (want.abs() + u.abs())
    norm = u.square().sum((1, 2)).sqrt()
    assert (off.square().sum((1, 2)).sqrt() <= 4e-3 * norm + near.square().sum((1, 2)).sqrt()).all()
    assert (off.abs() <= 1.5e-2 * norm[:, None, None] / (m * n) ** 0.5 + near).all()
    for p, w in zip(params, master):
        assert torch.equal(p, w.bfloat16())
