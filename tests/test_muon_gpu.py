"""Newton-Schulz orthogonalisation and the Muon step against their 64-bit
forms.

Tolerances. The products' operands are fp16, their sums fp32. Where an fp32
sum's error tips one fp16 rounding, the later steps amplify the difference, so
only the size of the error is predictable, not its bits: the 64-bit form with
fp16 operands, and the same with fp32 sums, both computed on the CPU, come out
1.2e-3 to 2.1e-3 off in norm for full-rank Gaussian matrices of 7 to 1,001
rows (4.2e-3 for 3 x 3, where one rounding is a ninth of all), at most 1.8e-2
of the result's rms off in one element, and a third of that for rank 16 under
1 % noise. Bounds: 3e-2 rms per element and, with the bf16 rounding of the
result (2^-8 of each element at most, 1.7e-3 in norm), 4e-3 in norm, 1e-2
below 16 rows."""
import math

import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import FsdpArgumentError, MuonHP, muon_step, newton_schulz, ops_wait_timeouts

pytestmark = pytest.mark.gpu


def _gauss(shape, seed, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g) * scale


ELEMENT = 3e-2


def _check(out, g, **kw):
    exact = ref.newton_schulz(g, **kw)
    rms = exact.square().mean().sqrt()
    bound = ref.BF16_U * exact.abs() + ELEMENT * rms + 1e-30
    bad = (out.double() - exact).abs() > bound
    assert not bad.any(), ((out.double() - exact).abs() / bound).max()
    norm = 4e-3 if min(g.shape) >= 16 else 1e-2
    assert (out.double() - exact).norm() <= norm * exact.norm() + 1e-30


SHAPES = [(1, 1, 1), (1, 1, 50), (1, 50, 1), (2, 2, 3), (3, 16, 16), (1, 64, 64), (1, 7, 200), (2, 200, 7),
          (1, 128, 128), (2, 129, 255), (1, 255, 129), (1, 256, 256), (2, 257, 300), (1, 300, 257), (1, 513, 1001),
          (1, 1001, 513), (5, 512, 512), (1, 384, 2048), (1, 2048, 384)]


@pytest.mark.parametrize("batch,m,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_newton_schulz(cuda_lib, batch, m, n, dtype):
    g = _gauss((batch, m, n), m * 3 + n).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    out = newton_schulz(g)
    assert out.shape == g.shape and out.dtype == torch.bfloat16
    for i in range(batch):
        _check(out[i], g[i])
    if batch == 1:
        assert torch.equal(newton_schulz(g[0]), out[0])
    assert ops_wait_timeouts() == 0


@pytest.mark.parametrize("batch,m,n", [(2, 7, 4099), (1, 300, 6001), (3, 5000, 20), (1, 2100, 256), (8, 3, 2500)])
def test_long_sums(cuda_lib, batch, m, n):
    """Few tiles and a long side: S is summed in parts."""
    g = _gauss((batch, m, n), m + n)
    out = newton_schulz(g)
    for i in range(batch):
        _check(out[i], g[i])
    assert torch.equal(newton_schulz(g), out)


@pytest.mark.parametrize("batch,k,l", [(1, 1, 1), (3, 1, 97), (28, 2, 2), (200, 4, 4), (100, 8, 8), (50, 16, 16),
                                       (45, 2, 1939), (8, 9, 2485), (3, 25, 504), (2, 31, 33), (2, 32, 32),
                                       (1, 32, 700), (2, 5, 30011)])
@pytest.mark.parametrize("tall", [False, True])
def test_thin_matrices(cuda_lib, batch, k, l, tall):
    """fp32 throughout: the 64-bit form with every product rounded to fp32
    (CPU, 300 square Gaussian matrices each of 4 to 32 rows, and rank 1 and 2
    under noise) is 7e-4 off in norm at most; the result's bf16 rounding is
    2^-8 of each element at most."""
    g = _gauss((batch, l, k) if tall else (batch, k, l), k + l)
    if k > 4:
        g[0] = (_gauss((l, 2), 1, 1.0) @ _gauss((2, k), 2, 1.0) if tall else _gauss((k, 2), 1, 1.0) @ _gauss((2, l), 2, 1.0)) + 10 * g[0]
    out = newton_schulz(g)
    for i in range(batch):
        exact = ref.newton_schulz(g[i])
        assert (out[i].double() - exact).norm() <= (ref.BF16_U + 1e-3) * exact.norm(), i
    assert torch.equal(newton_schulz(g), out)
    wide = torch.zeros(batch, g.shape[1] + 1, g.shape[2] + 3, device="cuda", dtype=torch.bfloat16)
    newton_schulz(g, out=wide[:, :-1, 1:-2])
    assert torch.equal(wide[:, :-1, 1:-2], out)
    wide[:, :-1, 1:-2] = 0
    assert not wide.any()


@pytest.mark.parametrize("m,n", [(3, 50), (50, 3), (16, 1600), (12, 4001), (4001, 12), (1, 40000)])
def test_thin_muon_step(cuda_lib, m, n):
    """As test_muon_step, with the bound of test_thin_matrices on the update."""
    grads, master, mom, params = _state(3, m, n, 3, torch.bfloat16, 7 + m)
    old_w, old_m = [w.clone() for w in master], [x.clone() for x in mom]
    muon_step(grads, master, mom, params, MuonHP(lr=0.02, momentum=0.9, weight_decay=0.1))
    for i in range(3):
        w, x, u = ref.muon(grads[i], old_w[i], old_m[i], 0.02, 0.9, 0.1, max(1.0, m / n) ** 0.5, True)
        size = sum(q.double().abs() for q in grads[i]) / 3 + old_m[i].double().abs()
        assert ((mom[i].double() - x).abs() <= 7 * 2 * ref.F32_U * size).all()
        err = (master[i].double() - w).norm()
        assert err <= 1e-3 * u.norm() + 4 * ref.F32_U * (w.norm() + u.norm())
        assert torch.equal(params[i], master[i].bfloat16())


def test_nearly_low_rank(cuda_lib):
    g = _gauss((512, 16), 1, 1.0) @ _gauss((16, 768), 2, 1.0) + 0.01 * _gauss((512, 768), 3, 1.0)
    _check(newton_schulz(g), g)
    _check(newton_schulz(g.t().contiguous()), g.t())


def test_singular_values_end_near_one(cuda_lib):
    s = torch.linalg.svdvals(newton_schulz(_gauss((200, 600), 4)).float())
    assert 0.6 < s.min() and s.max() < 1.3


@pytest.mark.parametrize("steps", [0, 1, 2, 7])
def test_steps_and_coefficients(cuda_lib, steps):
    g = _gauss((2, 130, 70), 5)
    out = newton_schulz(g, steps=steps, coefficients=(1.5, -0.5, 0.0), eps=1e-3)
    for i in range(2):
        _check(out[i], g[i], steps=steps, coef=(1.5, -0.5, 0.0), eps=1e-3)


def test_zeros_and_nan_keep_to_their_matrix(cuda_lib):
    g = _gauss((4, 40, 72), 6)
    clean = newton_schulz(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    out = newton_schulz(g)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert not out[1].any() and torch.isnan(out[2]).any()


def test_strides_streams_and_given_output(cuda_lib):
    big = _gauss((3, 2, 75, 61), 7)
    g = big[:, 1, :70, 3:53]  # batch and row strides wider than the matrix, odd start
    want = newton_schulz(g.contiguous())
    wide = torch.full((3, 73, 60), 9.0, device="cuda", dtype=torch.bfloat16)
    out = wide[:, :70, 5:55]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert newton_schulz(g, out=out, stream=s) is out
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    assert (wide[:, 70:] == 9).all() and (wide[:, :, :5] == 9).all() and (wide[:, :, 55:] == 9).all()


def _state(n_mats, m, n, R, dt, seed):
    grads = [[_gauss((m, n), seed + 31 * i + q).to(dt) for q in range(R)] for i in range(n_mats)]
    master = [_gauss((m, n), seed + 7 + i, 1 / math.sqrt(n)) for i in range(n_mats)]
    mom = [_gauss((m, n), seed + 77 + i) for i in range(n_mats)]
    return grads, master, mom, [w.bfloat16() for w in master]


@pytest.mark.parametrize("n_mats,m,n,R,dt", [(1, 64, 64, 1, torch.bfloat16), (3, 130, 257, 4, torch.bfloat16),
                                             (2, 513, 100, 8, torch.float32), (1, 1, 33, 2, torch.float32),
                                             (70, 24, 40, 2, torch.bfloat16), (1, 600, 1100, 3, torch.bfloat16)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step(cuda_lib, n_mats, m, n, R, dt, nesterov):
    """Momentum: two fp32 operations per element after the fold of R. Master:
    the update's own error (ELEMENT of its rms) and two fp32 operations."""
    grads, master, mom, params = _state(n_mats, m, n, R, dt, 100 + m)
    old_w, old_m = [w.clone() for w in master], [x.clone() for x in mom]
    hp = MuonHP(lr=0.02, momentum=0.9, weight_decay=0.1, nesterov=nesterov)
    muon_step(grads, master, mom, params, hp)
    scale = max(1.0, m / n) ** 0.5
    for i in range(n_mats):
        w, x, u = ref.muon(grads[i], old_w[i], old_m[i], 0.02, 0.9, 0.1, scale, nesterov)
        size = sum(q.double().abs() for q in grads[i]) / R + old_m[i].double().abs()
        assert ((mom[i].double() - x).abs() <= (R + 4) * 2 * ref.F32_U * size).all()
        bound = ELEMENT * u.square().mean().sqrt() + 4 * ref.F32_U * (w.abs() + u.abs())
        assert ((master[i].double() - w).abs() <= bound).all(), ((master[i].double() - w).abs() / bound).max()
        assert torch.equal(params[i], master[i].bfloat16())


def test_muon_without_params_and_mixed_shapes(cuda_lib):
    a, b = _state(2, 40, 72, 2, torch.float32, 5), _state(1, 72, 40, 2, torch.float32, 6)
    lists = [x + y for x, y in zip(a, b)]
    alone = [[w.clone() for w in part[1]] for part in (a, b)]
    alone_m = [[w.clone() for w in part[2]] for part in (a, b)]
    hp = MuonHP(lr=0.01)
    muon_step(lists[0], lists[1], lists[2], None, hp)
    for part, w, x in zip((a, b), alone, alone_m):
        muon_step(part[0], w, x, None, hp)
    for got, want in zip(lists[1], alone[0] + alone[1]):
        assert torch.equal(got, want)


def test_muon_zero_steps(cuda_lib):
    grads, master, mom, params = _state(2, 30, 50, 2, torch.bfloat16, 9)
    old_w, old_m = [w.clone() for w in master], [x.clone() for x in mom]
    muon_step(grads, master, mom, params, MuonHP(lr=0.1, steps=0))
    for i in range(2):
        w, _, u = ref.muon(grads[i], old_w[i], old_m[i], 0.1, 0.95, 0.0, 1.0, steps=0)
        assert ((master[i].double() - w).abs() <= 1e-5 * u.abs().max() + 4 * ref.F32_U * w.abs()).all()
        assert torch.equal(params[i], master[i].bfloat16())


def test_refusals(cuda_lib):
    g = _gauss((8, 16), 1)
    for bad in (lambda: newton_schulz(g.half()), lambda: newton_schulz(g.cpu()), lambda: newton_schulz(g[0]),
                lambda: newton_schulz(g.t()), lambda: newton_schulz(g, out=torch.empty_like(g)),
                lambda: newton_schulz(g[:0])):
        with pytest.raises(FsdpArgumentError):
            bad()
    for bad in (lambda: newton_schulz(g, steps=65), lambda: newton_schulz(g, eps=-1.0),
                lambda: newton_schulz(g, coefficients=(float("nan"), 0.0, 0.0))):
        with pytest.raises(Exception, match="fsdp_newton_schulz"):
            bad()
    grads, master, mom, params = _state(1, 8, 16, 2, torch.float32, 3)
    for args in (([], master, mom, params), (grads, master, mom, [params[0].float()]),
                 ([[grads[0][0], grads[0][1].bfloat16()]], master, mom, params),
                 (grads, [master[0][:, ::2]], mom, params), ([[]], master, mom, params)):
        with pytest.raises(FsdpArgumentError):
            muon_step(*args, MuonHP(lr=0.1))
    for hp in (MuonHP(lr=-1.0), MuonHP(lr=0.1, momentum=1.0), MuonHP(lr=0.1, update_scale=0.0)):
        with pytest.raises(Exception, match="hyper-parameters"):
            muon_step(grads, master, mom, params, hp)
    with pytest.raises(Exception, match="overlaps"):
        muon_step(grads, master, master, params, MuonHP(lr=0.1))
