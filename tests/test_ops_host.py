"""The operators' C ABI on the host (no GPU): every argument error is caught
before any CUDA call, with its status and message, and the workspace queries
answer without a device."""
import ctypes

import pytest

from fully_sharded_state_gb300 import build, capi

BASE = 1 << 40
MB = 1 << 20
OK, EINVAL, EALIGN, ERANGE, EUNSUP = (capi.FSDP_OK, capi.FSDP_EINVAL, capi.FSDP_EALIGN, capi.FSDP_ERANGE,
                                      capi.FSDP_EUNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def at(k):
    return BASE + k * 64 * MB


def call(fn, defaults, **over):
    return fn(*{**defaults, **over}.values())


NORM = dict(rows=8, cols=64, x=at(0), ldx=64, dtype=1, gamma=at(1), beta=at(2), pdtype=1, eps=1e-5, y=at(3), ldy=64,
            mean=at(4), rstd=at(5), stream=None)


@pytest.mark.parametrize("over,status,word", [
    (dict(rows=-1), EINVAL, b"rows"), (dict(cols=0), EINVAL, b"cols"), (dict(cols=1 << 32), ERANGE, b"cols"),
    (dict(dtype=7), EUNSUP, b"dtype"), (dict(pdtype=-1), EUNSUP, b"dtype"), (dict(eps=0.0), EINVAL, b"eps"),
    (dict(eps=float("nan")), EINVAL, b"eps"), (dict(mean=None), EINVAL, b"together"), (dict(x=None), EINVAL, b"x is"),
    (dict(x=at(0) + 1), EALIGN, b"x is"), (dict(ldx=63), EINVAL, b"x has"), (dict(y=at(0) + 128), EINVAL, b"overlaps"),
    (dict(gamma=None), EINVAL, b"gamma"), (dict(beta=at(4)), EINVAL, b"overlaps"),
    (dict(mean=at(4) + 2), EALIGN, b"mean")])
def test_layer_norm_refuses(lib, over, status, word):
    assert call(lib.fsdp_layer_norm, NORM, **over) == status
    assert word in lib.fsdp_last_error()


def test_layer_norm_of_no_rows_does_nothing(lib):
    assert call(lib.fsdp_layer_norm, NORM, rows=0, x=None, y=None, mean=None, rstd=None) == OK


BACK = dict(rows=8, cols=64, dy=at(0), lddy=64, x=at(1), ldx=64, dtype=0, gamma=at(2), pdtype=0, mean=at(3),
            rstd=at(4), dx=at(5), lddx=64, dgamma=at(6), dbeta=at(7), ws=at(8), bytes=64 * MB, stream=None)


@pytest.mark.parametrize("over,status,word", [
    (dict(cols=-3), EINVAL, b"cols"), (dict(dy=None), EINVAL, b"dy"), (dict(mean=None), EINVAL, b"mean"),
    (dict(dgamma=None), EINVAL, b"dgamma"), (dict(bytes=16), EINVAL, b"workspace"), (dict(ws=None), EINVAL, b"workspace"),
    (dict(ws=at(8) + 16), EALIGN, b"workspace"), (dict(dx=at(0)), EINVAL, b"overlaps"),
    (dict(dbeta=at(6) + 4), EINVAL, b"overlaps"), (dict(lddx=1), EINVAL, b"dx")])
def test_layer_norm_backward_refuses(lib, over, status, word):
    assert call(lib.fsdp_layer_norm_backward, BACK, **over) == status
    assert word in lib.fsdp_last_error()


LOSS = dict(rows=8, cols=64, vocab=100, hidden=at(0), ldh=64, weight=at(1), ldw=64, targets=at(2), ignore=-100,
            reduction=0, scale=1.0, loss=at(3), row_loss=at(4), dhidden=at(5), lddh=64, dweight=at(6), lddw=64,
            piece=0, ws=at(7), bytes=64 * MB, stream=None)


@pytest.mark.parametrize("over,status,word", [
    (dict(rows=-1), EINVAL, b"rows"), (dict(vocab=0), EINVAL, b"vocab"), (dict(vocab=1 << 40), ERANGE, b"vocab"),
    (dict(piece=-1), EINVAL, b"piece_rows"), (dict(reduction=2), EINVAL, b"reduction"),
    (dict(scale=float("inf")), EINVAL, b"grad_scale"), (dict(scale=1e300), EINVAL, b"grad_scale"),
    (dict(dhidden=None), EINVAL, b"together"), (dict(dweight=None), EINVAL, b"together"),
    (dict(targets=at(2) + 4), EALIGN, b"targets"), (dict(ldw=8), EINVAL, b"weight"), (dict(loss=None), EINVAL, b"loss"),
    (dict(dweight=at(1)), EINVAL, b"overlaps"), (dict(bytes=0), EINVAL, b"workspace")])
def test_linear_cross_entropy_refuses(lib, over, status, word):
    assert call(lib.fsdp_linear_cross_entropy, LOSS, **over) == status
    assert word in lib.fsdp_last_error()


SCHULZ = dict(batch=2, m=8, n=16, g=at(0), ldg=16, stride=128, dtype=1, out=at(1), ldo=16, ostride=128, steps=5,
              eps=1e-7, a=3.4445, b=-4.775, c=2.0315, ws=at(2), bytes=64 * MB, stream=None)


@pytest.mark.parametrize("over,status,word", [
    (dict(batch=-1), EINVAL, b"batch"), (dict(batch=70000), EINVAL, b"batch"), (dict(m=0), EINVAL, b"m ="),
    (dict(n=1 << 33), ERANGE, b"n ="), (dict(steps=-1), EINVAL, b"steps"), (dict(steps=65), EINVAL, b"steps"),
    (dict(eps=-1.0), EINVAL, b"eps"), (dict(b=float("inf")), EINVAL, b"coefficients"), (dict(dtype=3), EUNSUP, b"dtype"),
    (dict(stride=100), EINVAL, b"batch stride"), (dict(ldo=15), EINVAL, b"row stride"), (dict(out=at(0)), EINVAL, b"overlaps"),
    (dict(bytes=100), EINVAL, b"workspace")])
def test_newton_schulz_refuses(lib, over, status, word):
    assert call(lib.fsdp_newton_schulz, SCHULZ, **over) == status
    assert word in lib.fsdp_last_error()


def _muon(lib, n_mats=2, m=8, n=16, R=2, grads=None, dt=1, mom=None, master=None, params=None, hp=None, ws=at(40),
          nbytes=64 * MB, **hyper):
    arr = lambda k0, k: (ctypes.c_void_p * k)(*[at(k0 + i) for i in range(k)])  # noqa: E731
    h = dict(lr=0.1, momentum=0.9, weight_decay=0.0, eps=1e-7, update_scale=1.0, nesterov=1, steps=5, a=3.0, b=-4.0,
             c=2.0) | hyper
    s = capi.MuonHPStruct(*h.values())
    return lib.fsdp_muon(n_mats, m, n, R, grads or arr(0, 8), dt, mom or arr(10, 4), master or arr(20, 4),
                         params or arr(30, 4), None if hp is False else ctypes.byref(s), ws, nbytes, None)


@pytest.mark.parametrize("over,status,word", [
    (dict(n_mats=0), EINVAL, b"n_mats"), (dict(n_mats=65), EINVAL, b"n_mats"), (dict(R=0), EINVAL, b"R ="),
    (dict(R=65), EINVAL, b"R ="), (dict(n_mats=64, R=64), EINVAL, b"n_mats * R"), (dict(m=0), EINVAL, b"m ="),
    (dict(hp=False), EINVAL, b"hp"), (dict(lr=-1.0), EINVAL, b"hyper"), (dict(momentum=1.0), EINVAL, b"hyper"),
    (dict(update_scale=0.0), EINVAL, b"hyper"), (dict(weight_decay=float("nan")), EINVAL, b"hyper"),
    (dict(steps=100), EINVAL, b"steps"), (dict(dt=9), EUNSUP, b"dtype"), (dict(nbytes=1), EINVAL, b"workspace")])
def test_muon_refuses(lib, over, status, word):
    assert _muon(lib, **over) == status
    assert word in lib.fsdp_last_error()


def test_muon_refuses_buffers_that_overlap(lib):
    same = (ctypes.c_void_p * 4)(*[at(10 + i) for i in range(4)])
    assert _muon(lib, mom=same, master=same) == EINVAL
    assert b"overlaps" in lib.fsdp_last_error()
    odd = (ctypes.c_void_p * 4)(at(20), at(21) + 2, at(22), at(23))
    assert _muon(lib, master=odd) == EALIGN
    assert b"master[1]" in lib.fsdp_last_error()


def test_workspace_queries(lib):
    n = ctypes.c_int64(-1)
    q = ctypes.byref(n)
    for fn, sizes in ((lib.fsdp_layer_norm_backward_workspace, (1000, 513)),
                      (lib.fsdp_linear_cross_entropy_workspace, (1000, 513, 5001, 1, 0, 0)),
                      (lib.fsdp_linear_cross_entropy_workspace, (0, 8, 5, 0, 1, 0)),
                      (lib.fsdp_newton_schulz_workspace, (3, 100, 7)), (lib.fsdp_muon_workspace, (3, 100, 7))):
        assert fn(*sizes, q) == OK and n.value > 0 and n.value % 256 == 0 or fn is lib.fsdp_layer_norm_backward_workspace
        assert fn(*sizes, None) == EINVAL
        assert fn(*(-1,) + sizes[1:], q) == EINVAL
    # pieces of the rows bound the exponentials' share: 2 GiB by default
    big, small = [], []
    for rows in (16384, 65536, 262144):
        assert lib.fsdp_linear_cross_entropy_workspace(rows, 64, 128000, 1, 1, 0, q) == OK
        big.append(n.value)
        assert lib.fsdp_linear_cross_entropy_workspace(rows, 64, 128000, 1, 1, 1024, q) == OK
        small.append(n.value)
    assert big[2] < 2 * (1 << 31) and small[2] < 1 << 30 and big == sorted(big)


def test_timeout_count_refuses_bad_arguments(lib):
    n = ctypes.c_uint64(0)
    assert lib.fsdp_ops_wait_timeouts(-1, ctypes.byref(n)) == EINVAL
    assert lib.fsdp_ops_wait_timeouts(0, None) == EINVAL


def test_python_functions_refuse_host_tensors():
    import torch

    import fully_sharded_state_gb300 as fsdp
    x = torch.zeros(4, 8)
    t = torch.zeros(4, dtype=torch.int64)
    for bad in (lambda: fsdp.layer_norm(x, x[0]), lambda: fsdp.layer_norm_backward(x, x, x[0], x[:, 0], x[:, 0]),
                lambda: fsdp.linear_cross_entropy(x.bfloat16(), x.bfloat16(), t), lambda: fsdp.newton_schulz(x),
                lambda: fsdp.muon_step([[x]], [x], [x], None, fsdp.MuonHP(lr=0.1))):
        with pytest.raises(fsdp.FsdpArgumentError):
            bad()
