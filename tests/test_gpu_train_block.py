"""The operators together, as a training program uses them: norms forward and
backward under autograd, clipping over all gradients, Muon for the matrices,
AdamW with fp32 and 8-bit states for the rest."""

import math

import pytest
import torch

import memory_reduced_muon_gb300 as q

pytestmark = pytest.mark.gpu


def test_training_learns_and_repeats():
    from memory_reduced_muon_gb300 import train_block
    first, last, last8 = train_block.train(steps=150, rows=2048, seed=3)
    # at random: log 512; learned: the noise's entropy, 0.1 log 512 + H(0.1) = 0.95 or so
    assert abs(first - math.log(512)) < 1.0
    assert last < 2.0
    assert abs(last8 - last) < 0.05
    again = train_block.train(steps=150, rows=2048, seed=3)
    assert abs(again[1] - last) < 0.2      # torch's embedding gradient adds in no fixed order


def test_a_gradient_that_is_not_finite_leaves_adamw_parameters_alone():
    from memory_reduced_muon_gb300 import train_block
    model = train_block.Block(seed=1)
    x, y = next(train_block.batches(model.vocab, 256, 2))
    model.step(x, y)
    before = [t.clone() for t in (model.embed, model.head, *model.gains)]
    with torch.no_grad():
        model.head16[0, 0] = float("inf")
    model.step(x, y)
    assert torch.isnan(model.norm[1])
    for a, b in zip(before, (model.embed, model.head, *model.gains)):
        assert torch.equal(a, b)
    q.qmuon_sync_status(model.muon_ws)
