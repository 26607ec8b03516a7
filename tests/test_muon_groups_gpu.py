"""A Muon step over matrices of several shapes is several calls of the
library: it is refused before any of them, or not at all."""
import pytest
import torch

from fully_sharded_state_gb300 import FsdpArgumentError, MuonHP, muon_step, ops

pytestmark = pytest.mark.gpu


def _lists(shapes, R=2):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return ([[r(s) for _ in range(R)] for s in shapes], [r(s) for s in shapes], [r(s) for s in shapes],
            [r(s).bfloat16() for s in shapes])


def _refused(lists, error, match=None):
    everything = [t for part in lists[1:] for t in part]
    before = [t.clone() for t in everything]
    with pytest.raises(error, match=match):
        muon_step(*lists, MuonHP(lr=0.1))
    torch.cuda.synchronize()
    for now, was in zip(everything, before):
        assert torch.equal(now, was)


@pytest.mark.parametrize("a,b", [((8, 16), (16, 8)), ((40, 300), (300, 40)), ((64, 64), (64, 128))])
def test_an_overlap_in_a_later_group(cuda_lib, a, b):
    lists = _lists([a, b])
    lists[2][1] = lists[1][1]
    _refused(lists, FsdpArgumentError, r"overlaps")


def test_one_buffer_in_two_groups(cuda_lib):
    """The two views' updates would follow one another."""
    lists = _lists([(8, 16), (16, 8)])
    lists[1][1] = lists[1][0].view(16, 8)
    _refused(lists, FsdpArgumentError, r"master\[1\] overlaps master\[0\]|master\[0\] overlaps master\[1\]")
    lists = _lists([(8, 16), (16, 8)])
    lists[0][1][0] = lists[2][0].view(16, 8)
    _refused(lists, FsdpArgumentError, r"overlaps")


def test_one_matrix_twice_among_many(cuda_lib):
    """More matrices of one shape than a call takes."""
    lists = _lists([(4, 6)] * 70)
    lists[1][69] = lists[1][0]
    _refused(lists, FsdpArgumentError, r"overlaps")


def test_no_memory_for_a_later_group(cuda_lib, monkeypatch):
    lists = _lists([(8, 16), (300, 40)])
    real = ops._workspace_bytes
    monkeypatch.setattr(ops, "_workspace_bytes", lambda query, k, m, n: 1 << 50 if m == 300 else real(query, k, m, n))
    _refused(lists, RuntimeError)


def test_gradients_may_be_shared(cuda_lib):
    """Inputs alone may be one buffer: both views' results as if they were two."""
    lists = _lists([(8, 16), (16, 8)])
    lists[0][1] = [q.view(16, 8) for q in lists[0][0]]
    apart = [[q.clone() for q in x] if isinstance(x, list) else x.clone() for x in lists[0]], \
        [t.clone() for t in lists[1]], [t.clone() for t in lists[2]], [t.clone() for t in lists[3]]
    muon_step(*lists, MuonHP(lr=0.1))
    muon_step(*apart, MuonHP(lr=0.1))
    for one, two in zip(lists[1] + lists[2] + lists[3], apart[1] + apart[2] + apart[3]):
        assert torch.equal(one, two)
