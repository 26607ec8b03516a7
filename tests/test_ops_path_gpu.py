"""The operators with the shard engine: the Muon step of a ZeRO-3 unit, and
the example that trains a head with all of them."""
import importlib.util
import os

import pytest
import torch

import ops_reference as ref
from fully_sharded_state_gb300 import (FsdpArgumentError, MuonHP, ShardedUnit, ops_wait_timeouts)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pdt,gdt,R,shapes", [
    ("bf16", "bf16", 4, [(64, 48), (33, 7), (64, 48), (0, 5), (5, 3, 8)]),
    ("f32", "f32", 2, [(129, 40)]),
    ("bf16", "f32", 3, [(17, 130), (130, 17), (256, 256)]),
])
def test_muon_of_a_zero3_unit(cuda_lib, pdt, gdt, R, shapes):
    """Every parameter against its own 64-bit step (the tolerance of the
    orthogonal update: 3e-2 of its rms), the padding untouched."""
    U = ShardedUnit(shapes, R, "zero3", pdt, gdt)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(U.P, device="cuda", generator=gen) * 0.1
    U.shard_from_full(w)
    tg = torch.bfloat16 if gdt == "bf16" else torch.float32
    grads = [(torch.randn(U.P, device="cuda", generator=gen) * 1e-2).to(tg) for _ in range(R)]
    hp = MuonHP(lr=0.01, momentum=0.8, weight_decay=0.1)
    mom = [torch.zeros(s).cuda().double().reshape(s[0], -1) if min(s) else None for s in shapes]
    for step in (1, 2):
        before = [m.clone() for m in U.master]
        U.reduce_scatter_muon(grads, hp)
        assert U.step == step
        used = [torch.zeros(U.S, dtype=torch.bool, device="cuda") for _ in range(R)]
        for i, s in enumerate(shapes):
            if min(s) == 0:
                continue
            rows, n = s[0], torch.Size(s).numel()
            r, at, full = U.layout.param_owner(i), U.layout.param_shard_offset(i), U.layout.param_full_offset(i)
            used[r][at:at + n] = True
            old = before[r][at:at + n].view(rows, -1)
            scale = max(1.0, rows / (n // rows)) ** 0.5
            want, mom[i], u = ref.muon([g[full:full + n].view(rows, -1) for g in grads], old, mom[i], 0.01, 0.8, 0.1,
                                       scale)
            got = U.master[r][at:at + n].view(rows, -1)
            assert ((got.double() - want).abs() <= 3e-2 * u.square().mean().sqrt() + 1e-6 * want.abs()).all()
            assert ((U.m[r][at:at + n].view(rows, -1).double() - mom[i]).abs() <= 1e-5 * mom[i].abs().max()).all()
            if pdt == "bf16":
                assert torch.equal(U.param_shard[r][at:at + n], U.master[r][at:at + n].bfloat16())
        for r in range(R):
            assert torch.equal(U.master[r][~used[r]], before[r][~used[r]])


def test_muon_refuses_shards_and_vectors(cuda_lib):
    hp = MuonHP(lr=0.1)
    U = ShardedUnit([(8, 8)], 2, "per_param")
    with pytest.raises(FsdpArgumentError, match="zero3"):
        U.reduce_scatter_muon(U.alloc_grads(), hp)
    U = ShardedUnit([(8, 8), (8,)], 2, "zero3")
    with pytest.raises(FsdpArgumentError, match="vectors"):
        U.reduce_scatter_muon(U.alloc_grads(), hp)
    U = ShardedUnit([(8, 8)], 2, "zero3")
    with pytest.raises(FsdpArgumentError):
        U.reduce_scatter_muon(U.alloc_grads()[:1], hp)
    assert U.step == 0


def test_example_learns(cuda_lib):
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=40, rows=256, vocab=501)
    assert 5.5 < losses[0] < 7.0  # log 501 = 6.2
    assert losses[-1] < 0.5 * losses[0] and all(v == v for v in losses)
    assert ops_wait_timeouts() == 0
