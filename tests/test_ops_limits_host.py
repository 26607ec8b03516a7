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


BASE, MB = 1 << 40, 1 << 20


def at(k):
    return BASE + k * 64 * MB


@pytest.mark.parametrize("rows,ld", [(1 << 24, 1 << 40), (1 << 25, 1 << 39), ((1 << 30) + 1, (1 << 34) + 64), (MOST, 1 << 40)])
@pytest.mark.parametrize("which", ["x", "y"])
def test_row_strides_whose_ranges_wrap(lib, rows, ld, which):
    """rows * ld elements past 2^63 would come out as a small or negative range,
    which nothing overlaps."""
    ldx, ldy = (ld, 64) if which == "x" else (64, ld)
    # the other matrix is small enough to be named after this one
    args = [rows, 64, at(0), ldx, 1, at(1 << 20), None, 1, 1e-5, at(1 << 21), ldy, None, None, None]
    assert lib.fsdp_layer_norm(*args) == capi.FSDP_ERANGE
    assert f"{which} ".encode() in lib.fsdp_last_error() and b"too large" in lib.fsdp_last_error()


def test_batch_strides_whose_ranges_wrap(lib):
    rows, ld = 1 << 24, 1 << 40
    st = lib.fsdp_newton_schulz(2, rows, 8, at(0), ld, 8 * rows, 1, at(1), 8, 8 * rows, 5, 1e-7, 3.0, -4.0, 2.0, at(2), 64 * MB,
                                None)
    assert st == capi.FSDP_ERANGE and b"g " in lib.fsdp_last_error()


def test_the_loss_alone_keeps_to_its_pieces(lib):
    """What it keeps of a row, 8 bytes per 128 words, is bounded as the
    exponentials are: by 2 GiB, or by piece_rows."""
    n = ctypes.c_int64(0)

    def ask(rows, piece, grad=0, cols=64, vocab=200000):
        assert lib.fsdp_linear_cross_entropy_workspace(rows, cols, vocab, grad, 1, piece, ctypes.byref(n)) == capi.FSDP_OK
        return n.value

    own = lambda rows: rows * (64 * 2 + 4 + 4 + 4) + 4096  # noqa: E731  # hidden's copy, source, target, its logit
    for rows in (1 << 18, 1 << 20, 1 << 22):
        assert ask(rows, 0) <= (1 << 31) + own(rows)
        assert ask(rows, 1024) <= 1024 * 1563 * 8 + own(rows)
    assert ask(100, 0) <= 100 * 1563 * 8 + own(128)
    assert ask(1 << 18, 1024) < ask(1 << 18, 4096) < ask(1 << 18, 0)


def test_every_entry_of_the_operators_is_guarded():
    """What an entry calls may throw (set_error keeps a string): each runs its
    body where exceptions are caught."""
    import os
    import re

    source = open(os.path.join(build.CSRC, "fsdp_ops_capi.cpp")).read()
    body = source[source.index('extern "C" {'):]
    entries = re.split(r"^fsdp_status (?=fsdp_)", body, flags=re.M)[1:]
    assert len(entries) >= 10
    for e in entries:
        name = e[:e.index("(")]
        first = e[e.index("{") + 1:].split(";")[1].strip()
        assert first.startswith("return guarded(fn, [&]()"), name
