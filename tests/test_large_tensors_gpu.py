"""Tensors of more than 2^31 elements: the experts' products and dropout reach their
last rows, and no place a multiple of 2^32 elements off. Compared at the first and
last rows of every expert and at rows on both sides of 2^31 elements, against 64 bits;
tolerances as in test_grouped_linear_gpu.py and test_dropout_gpu.py."""
import pytest
import torch

import tuning_reference as tune
from fully_sharded_state_gb300 import dropout, grouped_linear, grouped_linear_backward, ops_wait_timeouts
from ops_reference import BF16_U, F32_U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_given_up(cuda_lib):
    yield
    assert ops_wait_timeouts() == 0
    torch.cuda.empty_cache()


def _rows(rows, cols, bounds):
    edge = (1 << 31) // cols
    at = [b + i for b in bounds for i in (-2, -1, 0, 1)] + [edge + i for i in range(-2, 3)]
    return torch.tensor(sorted({r for r in at if 0 <= r < rows}), device="cuda")


def _big(rows, cols, gen):
    t = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for part in t.split(1 << 16):
        part.normal_(generator=gen)
    return t


def _near(got, want, absolute, terms):
    bound = terms * 2.0 ** -23 * absolute + BF16_U * want.abs() + 1e-38
    assert ((got.double() - want).abs() <= bound).all()


def _expert_of(r, bounds):
    return torch.searchsorted(torch.tensor(bounds, device="cuda"), r, right=True) - 1


def _check_rows(got, x, w, at, bounds):
    """got = x w_e^T at these rows, 0 at those of no expert."""
    e = _expert_of(at, bounds)
    for i, r in enumerate(at.tolist()):
        if 0 <= e[i] < w.shape[0]:
            a, b = x[r].double(), w[e[i]].double()
            _near(got[r], b @ a, b.abs() @ a.abs(), x.shape[1])
        else:
            assert (got[r] == 0).all()


# x of 2^31 elements, y of them; rows on 16 bytes and not
@pytest.mark.parametrize("rows,n,k", [(530000, 40, 4096), (530000, 4096, 40), (530000, 24, 4095)])
def test_many_rows(rows, n, k):
    gen = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randn(3, n, k, device="cuda", generator=gen).bfloat16()
    x, dy = _big(rows, k, gen), _big(rows, n, gen)
    bounds = [0, 130000, 130001, rows - 70]
    offsets = torch.tensor(bounds, device="cuda")
    at = _rows(rows, max(n, k), bounds + [rows])
    y = grouped_linear(x, w, offsets)
    _check_rows(y, x, w, at, bounds)
    del y
    dx, dw = grouped_linear_backward(dy, x, w, offsets)
    _check_rows(dx, dy, w.transpose(1, 2), at, bounds)
    # a part of dW by sums of 64 bits
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        want, size = (torch.zeros(n, k, dtype=torch.float64, device="cuda") for _ in range(2))
        for a, b in zip(dy[lo:hi].split(1 << 14), x[lo:hi].split(1 << 14)):
            a, b = a.double(), b.double()
            want += a.t() @ b
            size += a.abs().t() @ b.abs()
        _near(dw[e], want, size, hi - lo)


def test_large_weights():
    gen = torch.Generator(device="cuda").manual_seed(1)
    experts, n, k, rows = 40, 8192, 6656, 77
    w = _big(experts * n, k, gen).view(experts, n, k)
    assert w.numel() > 1 << 31
    x, dy = _big(rows, k, gen), _big(rows, n, gen)
    bounds = [0] * 10 + [5] * 29 + [6, 77]
    offsets = torch.tensor(bounds, device="cuda")
    at = torch.tensor([0, 4, 5, 6, 40, 76], device="cuda")
    _check_rows(grouped_linear(x, w, offsets), x, w, at, bounds)
    dx, dw = grouped_linear_backward(dy, x, w, offsets)
    _check_rows(dx, dy, w.transpose(1, 2), at, bounds)
    for e in (0, 9, 37, 38, 39):
        a, b = dy[bounds[e]:bounds[e + 1]].double(), x[bounds[e]:bounds[e + 1]].double()
        _near(dw[e], a.t() @ b, a.abs().t() @ b.abs(), max(1, a.shape[0]))
    assert not dw[10:37].any()


# whole groups, units of 256 columns, narrow rows; the last with more than 2^31 elements of fp32
@pytest.mark.parametrize("rows,cols,dtype", [(530000, 4096, torch.bfloat16), (530000, 4095, torch.bfloat16),
                                             (40_000_000, 57, torch.bfloat16), (2_200_000, 1000, torch.float32)])
def test_dropout(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for part in x.split(1 << 16):
        part.normal_(generator=gen)
    y = dropout(x, 0.3, 7, offset=(1 << 40) + 3)
    for r in _rows(rows, cols, [0, rows]).tolist():
        # the generator for this row alone: its counter has the row in its second word
        keep_of = round(0.7 * 65536)
        group = range((cols + 7) // 8)
        words = [tune.philox([g, r, 3, 256], [7, 0]) for g in group]
        draws = torch.tensor([h for c in words for q in c for h in (q & 0xFFFF, q >> 16)][:cols], device="cuda")
        want = torch.where(draws < keep_of, x[r].double() * (65536 / keep_of), torch.zeros(cols, device="cuda", dtype=torch.float64))
        units = BF16_U if dtype == torch.bfloat16 else 0.0
        assert ((y[r].double() - want).abs() <= (units + 3 * F32_U) * want.abs()).all()
        assert torch.equal(y[r] != 0, (want != 0) & (x[r] != 0))
