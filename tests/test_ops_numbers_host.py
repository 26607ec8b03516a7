"""Hyper-parameters that fp32, in which the kernels take them, cannot hold are
refused on the host (no GPU)."""
import ctypes

import pytest

from fully_sharded_state_gb300 import build, capi

BASE, MB = 1 << 40, 1 << 20
EINVAL = capi.FSDP_EINVAL


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def at(k):
    return BASE + k * 64 * MB


@pytest.mark.parametrize("eps", [1e300, 1e-60, 5e-324, 3.5e38])
def test_layer_norm_eps(lib, eps):
    """1e-60 is 0 in fp32: rows of one value would have an infinite rstd."""
    assert lib.fsdp_layer_norm(8, 64, at(0), 64, 1, at(1), None, 1, eps, at(3), 64, None, None, None) == EINVAL
    assert b"eps" in lib.fsdp_last_error()


@pytest.mark.parametrize("over", [dict(eps=1e39), dict(eps=1e-60), dict(a=1e300), dict(b=-1e39), dict(c=3.5e38)])
def test_newton_schulz_numbers(lib, over):
    h = dict(eps=1e-7, a=3.4445, b=-4.775, c=2.0315) | over
    assert lib.fsdp_newton_schulz(2, 8, 16, at(0), 16, 128, 1, at(1), 16, 128, 5, *h.values(), at(2), 64 * MB, None) == EINVAL
    assert b"coefficients" in lib.fsdp_last_error()


@pytest.mark.parametrize("over", [dict(lr=1e39), dict(lr=1e30, update_scale=1e30), dict(lr=1e20, weight_decay=-1e20),
                                  dict(update_scale=1e300), dict(lr=1e300, weight_decay=1e300),
                                  dict(momentum=1.0 - 2.0 ** -40)])
def test_muon_numbers(lib, over):
    """Momentum has to be below 1 in fp32 as well."""
    arr = lambda k0, k: (ctypes.c_void_p * k)(*[at(k0 + i) for i in range(k)])  # noqa: E731
    h = dict(lr=0.1, momentum=0.9, weight_decay=0.0, eps=1e-7, update_scale=1.0, nesterov=1, steps=5, a=3.0, b=-4.0,
             c=2.0) | over
    s = capi.MuonHPStruct(*h.values())
    assert lib.fsdp_muon(2, 8, 16, 2, arr(0, 4), 1, arr(10, 2), arr(20, 2), arr(30, 2), ctypes.byref(s), at(40), 64 * MB,
                         None) == EINVAL
    assert b"hyper-parameters" in lib.fsdp_last_error()
