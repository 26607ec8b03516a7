"""Which kernels the operators' calls take, asked on the host (no GPU)."""
import ctypes
import re

GB300_SMS = 152


def _text(fn, *args):
    from fully_sharded_state_gb300 import build, capi
    build.build()
    f = getattr(capi.load(), fn)
    f.restype = ctypes.c_int
    buf = ctypes.create_string_buffer(1 << 20)
    status = f(*args, buf, ctypes.c_int64(len(buf)))
    assert status == 0, capi.load().fsdp_last_error().decode()
    return buf.value.decode().splitlines()


def _numbers(line):
    """'what: kind key 1 key 2' -> a dict of what, kind and the keys."""
    what, rest = line.split(": ", 1)
    d = {k: int(v) for k, v in re.findall(r"(\w+) (\d+)", rest)}
    d["what"], d["kind"] = what, rest.split()[0]
    return d


def newton_schulz(batch, m, n, ranks=0, steps=5, sms=GB300_SMS):
    i = ctypes.c_int64
    return [_numbers(q) for q in _text("fsdp_ops_plan_newton_schulz", i(batch), i(m), i(n), ranks, steps, sms)]


def linear_cross_entropy(rows, cols, vocab, grad=True, aligned=True, piece_rows=0, sms=GB300_SMS):
    i = ctypes.c_int64
    return [_numbers(q) for q in _text("fsdp_ops_plan_linear_cross_entropy", i(rows), i(cols), i(vocab), int(grad),
                                       int(aligned), i(piece_rows), sms)]
