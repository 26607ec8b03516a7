"""The largest sizes that the operators take, on the host (no GPU)."""
import ctypes

import pytest

from fully_sharded_state_gb300 import build, capi

MOST = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def _walk(vocab, segments, step=256 * 8, flight=4):
    """The largest column that a block of the loss's pass over the rows forms:
    `flight` steps from a thread's last column, or the last segment's end."""
    segment = (-(-vocab // segments) + 7) // 8 * 8
    cols = (vocab + 7) // 8 * 8
    return max(segments * segment, cols - 1 + flight * step)


@pytest.mark.parametrize("segments", [1, 7, 64, 8 * 152])
def test_columns_stay_in_32_bits(lib, segments):
    n = ctypes.c_int64(0)
    ask = lambda vocab: lib.fsdp_linear_cross_entropy_workspace(8, 8, vocab, 1, 1, 0, ctypes.byref(n))  # noqa: E731
    largest = max(v for v in (MOST, (1 << 31) - 8192, (1 << 31) - 1024) if ask(v) == capi.FSDP_OK)
    assert _walk(largest, segments) < 1 << 31
    assert ask(MOST) == capi.FSDP_OK and ask(MOST + 1) == capi.FSDP_ERANGE


@pytest.mark.parametrize("query,sizes", [("fsdp_layer_norm_backward_workspace", (1, 1)),
                                         ("fsdp_linear_cross_entropy_workspace", (1, 1, 1, 1, 1, 0)),
                                         ("fsdp_newton_schulz_workspace", (1, 1, 1)), ("fsdp_muon_workspace", (1, 1, 1))])
def test_every_size_has_the_limit(lib, query, sizes):
    n = ctypes.c_int64(0)
    for i in {"fsdp_layer_norm_backward_workspace": (0, 1), "fsdp_linear_cross_entropy_workspace": (0, 1, 2, 5),
              "fsdp_newton_schulz_workspace": (1, 2), "fsdp_muon_workspace": (1, 2)}[query]:
        at = lambda v: tuple(v if k == i else s for k, s in enumerate(sizes))  # noqa: E731
        assert getattr(lib, query)(*at(MOST), ctypes.byref(n)) == capi.FSDP_OK
        assert getattr(lib, query)(*at(MOST + 1), ctypes.byref(n)) == capi.FSDP_ERANGE
        assert b"too large" in lib.fsdp_last_error()
