"""A step of the training example whose gradients are not finite changes no
parameter and no state, of Muon's matrices or of AdamW's tensors."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _state(model):
    def tensors(x):
        if isinstance(x, torch.Tensor):
            return [x]
        if isinstance(x, (list, tuple)):
            return [t for y in x for t in tensors(y)]
        return tensors(getattr(x, "_keep", ()))     # a plan's arrays
    grads = {p.grad.data_ptr() for p in model.leaves}
    held = tensors([model.embed, model.head, *model.mats, *model.leaves, model.muon, model.adam, model.adam8])
    return [t for t in held if t.data_ptr() not in grads]


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_step_with_a_bad_gradient_changes_nothing(bad):
    from memory_reduced_muon_gb300 import train_block
    model = train_block.Block(seed=1)
    x, y = next(train_block.batches(model.vocab, 256, 2))
    model.step(x, y)
    head = model.head16.detach().clone()
    with torch.no_grad():
        model.head16[0, 0] = bad
    held = _state(model)
    assert len(held) >= 2 + 4 + 9 + 8 + 10     # masters, matrices, leaves, Muon's and AdamW's states
    before, t = [a.detach().clone() for a in held], model.t
    model.step(x, y)
    assert torch.isnan(model.norm[1])
    for a, b in zip(held, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))      # bits: one of them holds the bad value
    assert model.t == t
    # and training goes on
    with torch.no_grad():
        model.head16.copy_(head)
    assert math.isfinite(float(model.step(x, y)))
    assert model.t == t + 1
    assert all(bool(torch.isfinite(w).all()) for w in (model.embed, model.head, *model.mats, *model.gains))
    assert not torch.equal(model.mats[0], before[2])
    assert math.isfinite(float(model.step(x, y)))
