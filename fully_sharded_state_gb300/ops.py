"""The operators of a training step around a sharded unit.

``layer_norm`` and ``linear_cross_entropy_grad`` with their gradients, whose
outputs can be views of a unit's full gradient buffers; ``newton_schulz`` and
``muon_step``, the matrix-aware update that uses them. Each function checks
its tensors, allocates its outputs and workspace with torch on the stream
that the kernels run on, and makes one call of the CUDA library (C ABI in
``include/fsdp_ops.h``, where the formulas are); ``muon_step`` makes one per
shape, after all of its checks. Nothing synchronises.

Tensors are CUDA tensors of one device whose rows' elements are adjacent
(``stride(-1) == 1``); rows may be further apart. ``stream`` defaults to the
current stream of the tensors' device; tensors that another stream writes or
frees are the caller's to order, as everywhere in this package.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache

import torch

from . import capi
from .capi import FsdpArgumentError

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
_DT = {torch.bfloat16: capi.FSDP_BF16, torch.float32: capi.FSDP_F32}
_SAME = nullcontext()
NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _refuse(message):
    raise FsdpArgumentError(message)


def _matrix(t, name, rows=None, cols=None, dtype=None, device=None):
    """Checks a 2-D tensor; returns its row stride."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _refuse(f"{name} is not a CUDA tensor")
    shape = t.shape
    if len(shape) != 2:
        _refuse(f"{name} has {len(shape)} dimensions, needs 2")
    if device is not None and t.device != device:
        _refuse(f"{name} is on {t.device}, other tensors on {device}")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{name} has dtype {t.dtype}, needs {dtype}")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        _refuse(f"{name} has shape {tuple(shape)}, needs ({'any' if rows is None else rows}, "
                f"{'any' if cols is None else cols})")
    if r == 0 or c == 0:
        return c
    s0, s1 = t.stride()
    if s1 != 1 and c != 1:
        _refuse(f"{name}: the elements of a row are not adjacent")
    if r == 1:
        return c
    if s0 < c:
        _refuse(f"{name}: its rows overlap")
    return s0


def _vector(t, name, n, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _refuse(f"{name} is not a CUDA tensor")
    if t.device != device:
        _refuse(f"{name} is on {t.device}, other tensors on {device}")
    shape = t.shape
    if len(shape) != 1 or shape[0] != n:
        _refuse(f"{name} has shape {tuple(shape)}, needs ({n},)")
    if t.dtype != dtype:
        _refuse(f"{name} has dtype {t.dtype}, needs {dtype}")
    if n > 1 and t.stride(0) != 1:
        _refuse(f"{name} is not contiguous")
    return t.data_ptr()


def _on(stream, device):
    """The stream's handle, and the context in which memory is allocated for it."""
    if stream is None:
        # the handle alone: torch.cuda.current_stream() builds a Stream object, 2 us of a 25 us call
        return torch._C._cuda_getCurrentRawStream(device.index), _SAME
    return stream.cuda_stream, torch.cuda.stream(stream)


@lru_cache(maxsize=1024)
def _workspace_bytes(query, *sizes):
    """What the library's query `query` says for these sizes."""
    n = _i64(0)
    capi._check(getattr(capi.load(), query)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(query, *sizes, device):
    n = _workspace_bytes(query, *sizes)
    return torch.empty(n or 1, dtype=torch.uint8, device=device), n


def _ptr(t):
    return None if t is None else t.data_ptr()


# -- layer norm --------------------------------------------------------------------

def _norm_inputs(x, gamma):
    ldx = _matrix(x, "x")
    if not (x.dtype in _DT):
        _refuse(f"x has dtype {x.dtype}, needs bfloat16 or float32")
    if not (x.shape[1] > 0):
        _refuse("x has no columns")
    if not (isinstance(gamma, torch.Tensor) and gamma.dtype in _DT):
        _refuse("gamma needs dtype bfloat16 or float32")
    _vector(gamma, "gamma", x.shape[1], gamma.dtype, x.device)
    return ldx


def layer_norm(x, gamma, beta=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm of the rows of ``x`` [rows, cols]; ``beta`` None: no offset.
    Returns (y, mean, rstd): y in x's dtype (``out`` if given), the rows'
    statistics in fp32, which ``layer_norm_backward`` takes."""
    lib = capi.load()
    ldx = _norm_inputs(x, gamma)
    rows, cols = x.shape
    if beta is not None:
        _vector(beta, "beta", cols, gamma.dtype, x.device)
    handle, ctx = _on(stream, x.device)
    with ctx:
        y = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if out is None else out
        # two allocations: unbinding one costs 4 us more than the second
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    ldy = cols if out is None else _matrix(y, "out", rows, cols, x.dtype, x.device)
    capi._check(lib.fsdp_layer_norm(rows, cols, x.data_ptr(), ldx, _DT[x.dtype], gamma.data_ptr(), _ptr(beta),
                                    _DT[gamma.dtype], eps, y.data_ptr(), ldy, mean.data_ptr(),
                                    rstd.data_ptr(), handle))
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, with_beta: bool = True, dx=None, dgamma=None, dbeta=None,
                        stream=None):
    """The gradients of ``layer_norm`` from ``dy``: (dx, dgamma, dbeta). dgamma
    and dbeta have gamma's dtype; they can be given, e.g. as views of a unit's
    gradient buffer. dbeta is None where ``with_beta`` is false."""
    lib = capi.load()
    ldx = _norm_inputs(x, gamma)
    rows, cols = x.shape
    dev = x.device
    lddy = _matrix(dy, "dy", rows, cols, x.dtype, dev)
    pm = _vector(mean, "mean", rows, torch.float32, dev)
    pr = _vector(rstd, "rstd", rows, torch.float32, dev)
    handle, ctx = _on(stream, dev)
    lddx = cols if dx is None else _matrix(dx, "dx", rows, cols, x.dtype, dev)
    if dgamma is not None:
        _vector(dgamma, "dgamma", cols, gamma.dtype, dev)
    if dbeta is not None:
        if not with_beta:
            _refuse("dbeta is given, but with_beta is false")
        _vector(dbeta, "dbeta", cols, gamma.dtype, dev)
    with ctx:
        if dx is None:
            dx = torch.empty((rows, cols), dtype=x.dtype, device=dev)
        if dgamma is None:
            dgamma = torch.empty(cols, dtype=gamma.dtype, device=dev)
        if with_beta and dbeta is None:
            dbeta = torch.empty(cols, dtype=gamma.dtype, device=dev)
        ws, nws = _workspace("fsdp_layer_norm_backward_workspace", rows, cols, device=dev)
    capi._check(lib.fsdp_layer_norm_backward(
        rows, cols, dy.data_ptr(), lddy, x.data_ptr(), ldx, _DT[x.dtype], gamma.data_ptr(), _DT[gamma.dtype], pm, pr,
        dx.data_ptr(), lddx, dgamma.data_ptr(), _ptr(dbeta), ws.data_ptr(), nws, handle))
    return dx, dgamma, dbeta


# -- the loss of a linear head -----------------------------------------------------

def _loss_call(hidden, weight, targets, ignore_index, reduction, grad, grad_scale, dhidden, dweight, piece_rows,
               stream):
    lib = capi.load()
    ldh = _matrix(hidden, "hidden", dtype=torch.bfloat16)
    rows, cols = hidden.shape
    dev = hidden.device
    ldw = _matrix(weight, "weight", None, cols, torch.bfloat16, dev)
    vocab = weight.shape[0]
    if not (cols > 0 and vocab > 0):
        _refuse("hidden and weight need at least one column and one row")
    if not (reduction in ("mean", "sum")):
        _refuse(f"reduction {reduction!r} is not 'mean' or 'sum'")
    pt = _vector(targets, "targets", rows, torch.int64, dev)
    handle, ctx = _on(stream, dev)
    with ctx:
        loss = torch.empty((), dtype=torch.float32, device=dev)
        row_loss = torch.empty(rows, dtype=torch.float32, device=dev)
        if grad:
            lddh = cols if dhidden is None else _matrix(dhidden, "dhidden", rows, cols, torch.bfloat16, dev)
            lddw = cols if dweight is None else _matrix(dweight, "dweight", vocab, cols, torch.bfloat16, dev)
            if dhidden is None:
                dhidden = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
            if dweight is None:
                dweight = torch.empty((vocab, cols), dtype=torch.bfloat16, device=dev)
        else:
            lddh = lddw = cols
        aligned = int(weight.data_ptr() % 16 == 0 and ldw % 8 == 0)
        ws, nws = _workspace("fsdp_linear_cross_entropy_workspace", rows, cols, vocab, int(grad), aligned, piece_rows,
                             device=dev)
    capi._check(lib.fsdp_linear_cross_entropy(
        rows, cols, vocab, hidden.data_ptr(), ldh, weight.data_ptr(), ldw, pt, int(ignore_index),
        0 if reduction == "mean" else 1, float(grad_scale), loss.data_ptr(), row_loss.data_ptr(), _ptr(dhidden), lddh,
        _ptr(dweight), lddw, piece_rows, ws.data_ptr(), nws, handle))
    return loss, row_loss, dhidden, dweight


def linear_cross_entropy(hidden, weight, targets, ignore_index: int = -100, reduction: str = "mean", stream=None,
                         piece_rows: int = 0):
    """Cross entropy of ``hidden`` [rows, cols] @ ``weight`` [vocab, cols]^T
    against ``targets`` (int64), without the logits: (loss, row_loss), fp32.
    Rows whose target is ``ignore_index`` count for nothing. ``piece_rows`` as
    in ``linear_cross_entropy_grad``."""
    return _loss_call(hidden, weight, targets, ignore_index, reduction, False, 1.0, None, None, int(piece_rows),
                      stream)[:2]


def linear_cross_entropy_grad(hidden, weight, targets, ignore_index: int = -100, reduction: str = "mean",
                              grad_scale: float = 1.0, dhidden=None, dweight=None, piece_rows: int = 0, stream=None):
    """``linear_cross_entropy`` and its gradients times ``grad_scale``:
    (loss, row_loss, dhidden, dweight), the gradients in bf16. ``dweight`` can
    be a view of a unit's gradient buffer. ``piece_rows`` bounds the rows that
    are worked on at a time, and with them the workspace (0: 2 GiB of it)."""
    return _loss_call(hidden, weight, targets, ignore_index, reduction, True, grad_scale, dhidden, dweight,
                      int(piece_rows), stream)


# -- Newton-Schulz and Muon ----------------------------------------------------------

def newton_schulz(g, steps: int = 5, eps: float = 1e-7, coefficients=NEWTON_SCHULZ_COEFFICIENTS, out=None,
                  stream=None):
    """Orthogonalises ``g`` [m, n], or each matrix of [batch, m, n], by
    Newton-Schulz iteration; returns bf16 of the same shape. With the default
    coefficients and steps the singular values end between about 0.7 and 1.2."""
    lib = capi.load()
    if not (isinstance(g, torch.Tensor) and g.is_cuda):
        _refuse("g is not a CUDA tensor")
    if not (g.dtype in _DT):
        _refuse(f"g has dtype {g.dtype}, needs bfloat16 or float32")
    if not (g.dim() in (2, 3)):
        _refuse(f"g has {g.dim()} dimensions, needs 2 or 3")
    handle, ctx = _on(stream, g.device)
    with ctx:
        if out is None:
            out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
        g3 = g if g.dim() == 3 else g.unsqueeze(0)
        batch, m, n = g3.shape
        if not (m > 0 and n > 0):
            _refuse("g has no rows or no columns")
        ws, nws = _workspace("fsdp_newton_schulz_workspace", batch, m, n, device=g.device)
    if not (isinstance(out, torch.Tensor) and out.shape == g.shape and out.dtype == torch.bfloat16 and out.device == g.device):
        _refuse(f"out needs shape {tuple(g.shape)}, bfloat16, on {g.device}")
    o3 = out if out.dim() == 3 else out.unsqueeze(0)
    if batch == 0:
        return out
    ldg = _matrix(g3[0], "g")
    ldo = _matrix(o3[0], "out")
    a, b, c = coefficients
    capi._check(lib.fsdp_newton_schulz(batch, m, n, g.data_ptr(), ldg, g3.stride(0), _DT[g.dtype], out.data_ptr(), ldo,
                                       o3.stride(0), steps, eps, a, b, c, ws.data_ptr(), nws, handle))
    return out


@dataclass
class MuonHP:
    """Hyper-parameters of ``muon_step``. ``update_scale`` multiplies ``lr`` in
    the update; None: sqrt(max(1, m / n)) of an [m, n] matrix."""
    lr: float
    momentum: float = 0.95
    weight_decay: float = 0.0
    nesterov: bool = True
    eps: float = 1e-7
    update_scale: float | None = None
    steps: int = 5
    coefficients: tuple = NEWTON_SCHULZ_COEFFICIENTS

    def _c(self, m, n):
        scale = self.update_scale if self.update_scale is not None else max(1.0, m / n) ** 0.5
        return capi.MuonHPStruct(self.lr, self.momentum, self.weight_decay, self.eps, scale, int(self.nesterov),
                                 self.steps, *self.coefficients)


def muon_step(grads, master, momentum, params, hp: MuonHP, stream=None) -> None:
    """One Muon step of a list of matrices, in place. ``grads[i]``: the R
    ranks' gradients of matrix i (bf16 or fp32), folded in rank order and
    averaged; ``master[i]``, ``momentum[i]``: fp32; ``params``: None, or bf16
    matrices that receive the rounded master. Matrices of one shape go through
    the kernels together."""
    lib = capi.load()
    count = len(master)
    if not (len(grads) == count and len(momentum) == count and (params is None or len(params) == count)):
        _refuse(f"grads, master, momentum and params need one entry per matrix ({count})")
    groups = {}
    for i, w in enumerate(master):
        if not (isinstance(w, torch.Tensor) and w.is_cuda and w.dim() == 2):
            _refuse(f"master[{i}] is not a 2-D CUDA tensor")
        if not (len(grads[i]) > 0):
            _refuse(f"grads[{i}] is empty")
        groups.setdefault((w.shape[0], w.shape[1], len(grads[i]), grads[i][0].dtype), []).append(i)
    if not groups:
        return
    dev = master[0].device

    def ptr(t, m, n, dtype, name, *index):
        if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.shape == (m, n) and
                t.device == dev and t.is_contiguous()):
            return t.data_ptr()
        name += "".join(f"[{i}]" for i in index)
        _matrix(t, name, m, n, dtype, dev)
        _refuse(f"{name} is not contiguous")

    calls = []
    for (m, n, R, dt), ids in groups.items():
        if not (m > 0 and n > 0):
            _refuse("a matrix has no rows or no columns")
        if not (dt in _DT):
            _refuse(f"grads have dtype {dt}, need bfloat16 or float32")
        if not (R <= capi.FSDP_MAX_RANKS):
            _refuse(f"{R} ranks, at most {capi.FSDP_MAX_RANKS}")
        per = min(capi.FSDP_MUON_MAX_MATRICES, 1024 // R)
        for lo in range(0, len(ids), per):
            part = ids[lo:lo + per]
            k = len(part)
            g = (_vp * (k * R))(*[ptr(t, m, n, dt, "grads", i, q) for i in part for q, t in enumerate(grads[i])])
            mo = (_vp * k)(*[ptr(momentum[i], m, n, torch.float32, "momentum", i) for i in part])
            ma = (_vp * k)(*[ptr(master[i], m, n, torch.float32, "master", i) for i in part])
            po = None if params is None else (_vp * k)(*[ptr(params[i], m, n, torch.bfloat16, "params", i)
                                                         for i in part])
            calls.append((part, m, n, R, g, dt, mo, ma, po))
    if len(calls) > 1:
        _apart(calls)  # one call sees to its own
    # the workspace before the first launch, too; the calls follow one another in it
    handle, ctx = _on(stream, dev)
    nws = max(_workspace_bytes("fsdp_muon_workspace", len(part), m, n) for part, m, n, *_ in calls)
    with ctx:
        ws = torch.empty(nws or 1, dtype=torch.uint8, device=dev)
    for part, m, n, R, g, dt, mo, ma, po in calls:
        c = hp._c(m, n)
        capi._check(lib.fsdp_muon(len(part), m, n, R, g, _DT[dt], mo, ma, po, ctypes.byref(c), ws.data_ptr(), nws, handle))


def _apart(calls):
    """Refuses a matrix that is written and shares memory with another one, over
    all calls of a step: what each call checks of its own matrices."""
    spans = []
    for part, m, n, R, g, dt, mo, ma, po in calls:
        numel = m * n
        spans += [(p, p + numel * dt.itemsize, False, "grads", part[j // R], j % R) for j, p in enumerate(g)]
        for name, pointers, size in (("momentum", mo, 4), ("master", ma, 4), ("params", po or (), 2)):
            spans += [(p, p + numel * size, True, name, part[j], None) for j, p in enumerate(pointers)]
    spans.sort()
    name = lambda s: f"{s[3]}[{s[4]}]" + ("" if s[5] is None else f"[{s[5]}]")  # noqa: E731
    furthest = written = (0, 0)  # of all before, and of those that are written
    for s in spans:
        hit = furthest if s[2] else written
        if s[0] < hit[1]:
            _refuse(f"{name(s)} overlaps {name(hit)}")
        if s[1] > furthest[1]:
            furthest = s
        if s[2] and s[1] > written[1]:
            written = s


def ops_wait_timeouts(device=None) -> int:
    """Thread blocks of the matrix kernels on ``device`` (default: the current
    CUDA device) that gave up a wait since the library was loaded; 0 in every
    valid run. Synchronises the device."""
    n = ctypes.c_uint64(0)
    capi._check(capi.load().fsdp_ops_wait_timeouts(capi._device_index(device), ctypes.byref(n)))
    return int(n.value)
