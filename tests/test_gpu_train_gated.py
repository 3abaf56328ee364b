"""The embedding, the norm, the gated block and its 8-bit checkpoints together,
as the training example runs them: its gradients against the same model in
fp64, and its steps.

Roundings to bf16 (2^-8 of a value at most) lie one behind another: the sum, y,
h, the MLP's output, the next norm's sum and output, the logits; backward the
gradients at the same places, and dgate and dup.  Each moves what follows by
about as much relative to its norm, 14 of them by 14 2^-8 = 5.5%.  The
checkpoints move gate, up and y by 2^-4 of a value at most, which a gradient
takes on once each through up, y and act (the slope of silu, whose values lie
within [-0.1, 1.1], changes by less than 0.5 2^-4 |gate|): three times 2^-4 at
most if all erred alike and to their limits, 19%."""

import pytest
import torch
import torch.nn.functional as F

import memory_reduced_muon_gb300 as q

pytestmark = pytest.mark.gpu


def _reference(model, tokens, targets):
    """(loss, gradients of the leaves) in fp64, from the model's 16-bit weights."""
    from memory_reduced_muon_gb300.train_block import EPS
    leaves = [p.detach().double().requires_grad_(True) for p in model.leaves]
    embed, head, rest = leaves[0], leaves[1], leaves[2:]
    mats, gains = rest[:len(model.mats)], rest[len(model.mats):]
    norm = lambda x, g: x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * g   # noqa: E731
    x, stream = F.embedding(tokens, embed), 0.0
    for i in range(len(mats) // 3):
        stream = stream + x
        y = norm(stream, gains[i])
        x = (F.silu(y @ mats[3 * i].T) * (y @ mats[3 * i + 1].T)) @ mats[3 * i + 2].T
    loss = F.cross_entropy(norm(stream + x, gains[-1]) @ head.T, targets)
    loss.backward()
    return float(loss.detach()), [p.grad for p in leaves]


@pytest.mark.parametrize("rows", [1, 129, 2048])
def test_gradients_of_the_gated_model(rows):
    from memory_reduced_muon_gb300 import train_block
    model = train_block.Block(seed=5, gated=True)
    x, y = next(train_block.batches(model.vocab, rows, 6))
    for p in model.leaves:
        p.grad.zero_()
    loss = model.loss(x, y)
    loss.backward()
    want, grads = _reference(model, x, y)
    assert abs(float(loss.detach()) - want) <= 14 * 2.0 ** -8 * (1 + abs(want))
    for p, g in zip(model.leaves, grads):
        assert float((p.grad.double() - g).norm()) <= (14 * 2.0 ** -8 + 3 * 2.0 ** -4) * float(g.norm())


def test_gradients_repeat_bit_for_bit():
    from memory_reduced_muon_gb300 import train_block
    model = train_block.Block(seed=5, gated=True)
    x, y = next(train_block.batches(model.vocab, 1000, 6))
    runs = []
    for _ in range(2):
        for p in model.leaves:
            p.grad.zero_()
        stream, out = model.hidden(x)
        (stream.float().square().sum() + out.float().square().sum()).backward()
        runs.append([p.grad.clone() for p in (model.embed16, *model.mats16, *model.gains[:-1])])
    for a, b in zip(*runs):
        assert bool((a != 0).any()) and torch.equal(a, b)


def test_steps_of_the_gated_model_run():
    from memory_reduced_muon_gb300 import train_block
    model = train_block.Block(seed=2, gated=True)
    data = train_block.batches(model.vocab, 2048, 3)
    before = [m.clone() for m in (model.embed, *model.mats)]
    for _ in range(3):
        assert bool(torch.isfinite(model.step(*next(data))))
    q.qmuon_sync_status(model.muon_ws)
    for a, b in zip(before, (model.embed, *model.mats)):
        assert bool(torch.isfinite(b).all()) and not torch.equal(a, b)
    x, y = next(data)
    assert bool(torch.isfinite(model.loss_mxfp8(x, y)))
