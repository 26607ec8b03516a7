"""The kernels that the operators' calls take, on the host: every product has
a shape that the instruction has, whatever the sizes."""
import random

import ops_plan


def _sizes(rng, most):
    return int(round(most ** rng.random()))


def _check_products(plan, sizes):
    for p in plan:
        if p["kind"] != "product":
            continue
        # tcgen05.mma, 16-bit operands: N is a multiple of 16 up to 256 with the
        # 128 rows of one CTA, of 32 with the 256 of a pair
        assert p["columns"] % (16 * p["ctas"]) == 0 and 0 < p["columns"] <= p["tile"] <= 256, (sizes, p)


def test_products_of_the_loss_have_valid_shapes():
    rng = random.Random(0)
    cases = [(1001, 513, 50021), (1, 512, 32000), (256, 512, 32000), (8192, 4096, 65536), (300, 513, 777),
             (128, 72, 257), (1000, 264, 3001), (700, 96, 20011), (2, 1, 1)]
    cases += [(_sizes(rng, 16384), _sizes(rng, 8192), _sizes(rng, 200000)) for _ in range(400)]
    for case in cases:
        for grad, aligned, piece in ((True, True, 0), (True, False, 0), (True, True, 100), (False, True, 0)):
            plan = ops_plan.linear_cross_entropy(*case, grad=grad, aligned=aligned, piece_rows=piece)
            assert plan
            _check_products(plan, case)


def test_products_of_newton_schulz_have_valid_shapes():
    rng = random.Random(1)
    cases = [(1, 14336, 4096), (48, 512, 512), (3, 1001, 513), (1, 300, 6001), (3, 5000, 20), (1, 8192, 8192)]
    cases += [(_sizes(rng, 64), _sizes(rng, 8192), _sizes(rng, 8192)) for _ in range(400)]
    for case in cases:
        for ranks in (0, 3):
            _check_products(ops_plan.newton_schulz(*case, ranks=ranks), case)


def test_a_step_of_each_form():
    thin, = ops_plan.newton_schulz(64, 8, 512)
    assert thin["what"] == "newton_schulz (thin)"
    team, = ops_plan.newton_schulz(4, 512, 512, ranks=4)
    assert team["kind"] == "team" and team["what"] == "muon" and team["rounds"] == 1
    plan = ops_plan.newton_schulz(48, 512, 512, steps=2)
    assert [p["what"].split(" ", 1)[1] for p in plan] == ["(start)", "(scale)"] + ["(S)", "(P)", "(x)"] * 2


def _in_parts(*case):
    return any("S, parts" in p["what"] for p in ops_plan.newton_schulz(*case))


def test_sums_are_cut_where_that_is_shorter():
    """Times of five steps, in parts and whole, us: 1 x 300 x 6001 292 and 201,
    4 x 256 x 3000 240 and 166, 1 x 400 x 6000 366 and 223, 8 x 160 x 2048 168 and
    139; 8 x 33 x 14000 189 and 356, 1 x 128 x 14000 224 and 314, 1 x 400 x 40000 532
    and 890."""
    for case in ((1, 300, 6001), (1, 6001, 300), (4, 256, 3000), (4, 3000, 256), (1, 400, 6000), (8, 160, 2048), (8, 2048, 160)):
        assert not _in_parts(*case), case
    for case in ((20, 33, 6000), (8, 33, 14000), (1, 33, 40000), (1, 64, 14000), (1, 128, 14000), (1, 400, 40000), (1, 40000, 400)):
        assert _in_parts(*case), case
