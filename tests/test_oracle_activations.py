"""Pins of the embedding, gated feed-forward and checkpoint definitions (CPU only)."""

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import activations as act

RNG = np.random.default_rng


def _t(x):
    return torch.from_numpy(np.array(x, dtype=np.float64)).requires_grad_(True)


def test_embedding_matches_torch():
    r = RNG(1)
    table, tokens = _t(r.standard_normal((11, 5))), r.integers(0, 11, 40)
    out = F.embedding(torch.from_numpy(tokens), table) * 2.5
    np.testing.assert_allclose(act.embedding64(table.detach().numpy(), tokens, 2.5), out.detach().numpy(), rtol=1e-14)
    dout = r.standard_normal((40, 5))
    out.backward(torch.from_numpy(dout))
    grad, mag, count = act.embedding_grad64(dout, tokens, 11, 2.5)
    np.testing.assert_allclose(grad, table.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert count.sum() == 40 and (mag >= np.abs(grad) - 1e-12).all()


def test_tokens_outside_are_no_tokens():
    r = RNG(2)
    table, tokens = r.standard_normal((4, 3)), np.array([0, -1, 4, 3, 1 << 40])
    out = act.embedding64(table, tokens)
    assert (out[[1, 2, 4]] == 0).all() and (out[0] == table[0]).all() and (out[3] == table[3]).all()
    _, _, count = act.embedding_grad64(r.standard_normal((5, 3)), tokens, 4)
    assert count.tolist() == [1, 0, 0, 1]


_TORCH = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda x: F.gelu(x, approximate="tanh")}


@pytest.mark.parametrize("name", sorted(_TORCH))
def test_activations_match_torch(name):
    g = _t(np.concatenate([np.linspace(-30, 30, 4001), [0.0, 1e-12]]))
    y = _TORCH[name](g)
    y.sum().backward()
    a, slope = act.act64(name, g.detach().numpy())
    np.testing.assert_allclose(a, y.detach().numpy(), rtol=1e-9, atol=1e-13)
    np.testing.assert_allclose(slope, g.grad.numpy(), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("name", sorted(_TORCH))
def test_block_matches_autograd_and_differences(name):
    r = RNG(3)
    x, wg, wu = _t(r.standard_normal((6, 5))), _t(r.standard_normal((7, 5))), _t(r.standard_normal((7, 5)))
    h = _TORCH[name](x @ wg.T) * (x @ wu.T)
    dh = r.standard_normal((6, 7))
    h.backward(torch.from_numpy(dh))
    X, G, U = (v.detach().numpy() for v in (x, wg, wu))
    got, gate, up = act.gated_ffn64(X, G, U, name)
    np.testing.assert_allclose(got, h.detach().numpy(), rtol=1e-10, atol=1e-12)
    dgate, dup, again = act.gated_slopes64(dh, gate, up, name)
    np.testing.assert_allclose(again, got, rtol=0, atol=0)
    grads = act.gated_products64(dgate, dup, X, G, U)
    for a, b in zip(grads, (x, wg, wu)):
        np.testing.assert_allclose(a, b.grad.numpy(), rtol=1e-9, atol=1e-11)
    # against differences, along one random direction per array
    eps = 1e-6
    for k, grad in enumerate(grads):
        d = r.standard_normal(grad.shape)
        at = lambda s: np.sum(dh * act.gated_ffn64(*[v + s * d if i == k else v for i, v in enumerate((X, G, U))], name)[0])   # noqa: E731
        assert abs((at(eps) - at(-eps)) / (2 * eps) - np.sum(grad * d)) <= 1e-7 * (1 + np.abs(grad * d).sum())


def test_checkpoint_codec_round_trip():
    r = RNG(4)
    x = (r.standard_normal((9, 96)) * np.exp(r.uniform(-20, 20, (9, 96)))).astype(np.float32)
    x[3, 32:64] = 0.0
    payload, scale = act.encode(x)
    back = act.decode64(payload, scale)
    unit = np.repeat(2.0 ** (scale.astype(np.float64) - 127), 32, 1)
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * unit)).all()
    again = act.encode(back.astype(np.float32))
    np.testing.assert_array_equal(act.decode64(*again), back)
