"""Pins of the clipping, AdamW and RMS norm definitions (CPU only)."""

import numpy as np
import pytest
import torch

from oracle import carrier, training

RNG = np.random.default_rng


def test_clip_matches_torch():
    r = RNG(1)
    gs = [r.standard_normal(n) for n in (1, 7, 4096)]
    ps = [torch.nn.Parameter(torch.zeros(g.size, dtype=torch.float64)) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.from_numpy(g.copy())
    norm, coef = training.clip64(gs, 3.0)
    got = torch.nn.utils.clip_grad_norm_(ps, 3.0)
    assert abs(float(got) - norm) <= 1e-12 * norm
    np.testing.assert_allclose(ps[2].grad.numpy(), gs[2] * coef, rtol=1e-12)
    assert training.clip64(gs, 1e9)[1] == 1.0
    assert np.isnan(training.clip64([np.array([np.inf])], 1.0)[1])


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_adamw_matches_torch(wd):
    r = RNG(2)
    p0 = r.standard_normal(1000)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=wd)
    q, m, v = p0.copy(), np.zeros(1000), np.zeros(1000)
    for t in range(1, 6):
        g = r.standard_normal(1000)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        q, m, v = training.adamw64(q, g, m, v, t, 3e-3, 0.9, 0.95, 1e-8, wd)
    np.testing.assert_allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_e4m3_encoders_agree_with_torch():
    r = RNG(3)
    x = np.concatenate([r.standard_normal(20000) * np.exp(r.uniform(-12, 5, 20000)), [0.0, 448.0, -448.0, 2.0 ** -9]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(carrier.e4m3_encode(x), want)
    # a value on the grid stays whatever the random bits are; others go to one of their two neighbours
    on = carrier.e4m3_decode(np.arange(0x7F, dtype=np.uint8)).astype(np.float32)
    for u in (0, 1, 40000, 65535):
        np.testing.assert_array_equal(training.e4m3_stochastic(on, np.full(on.size, u)), np.arange(0x7F))
    lo = training.e4m3_stochastic(x, np.zeros(x.size, dtype=np.int64))
    hi = training.e4m3_stochastic(x, np.full(x.size, 65535))
    vlo, vhi = (np.abs(carrier.e4m3_decode(c)) for c in (lo, hi))
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    # the largest offset, 65535/65536 of a step, leaves down only what lies within the last 1/65536 above the grid
    assert (vlo <= np.abs(x)).all() and (vhi >= np.abs(x) - step * 2.0 ** -16).all()
    assert (hi.astype(int) - lo.astype(int) <= 1).all()


def test_stochastic_rounding_is_unbiased():
    r = RNG(4)
    x = np.float32([0.3, 1.1, 17.3, 0.004, 0.0007])
    n = 200000
    for v in x:
        u = r.integers(0, 65536, n)
        q = carrier.e4m3_decode(training.e4m3_stochastic(np.full(n, v, np.float32), u))
        step = 2.0 ** (max(np.floor(np.log2(v)), -6) - 3)
        # a coin of two values one step apart: standard error at most step / (2 sqrt(n)); 5 of them
        assert abs(q.mean() - v) <= 5 * step / (2 * np.sqrt(n)) + step * 2.0 ** -16


def test_e4m3_adamw_tracks_fp64_and_keeps_zero_blocks():
    r = RNG(5)
    n = 1000
    g = r.standard_normal(n).astype(np.float32) * 1e-2
    g[256:512] = 0.0
    p = r.standard_normal(n).astype(np.float32)
    z, zb = np.zeros(n, np.uint8), np.zeros(4, np.float32)
    p1, m1, v1, mm, vm = training.adamw_e4m3(p, g, z, z, zb, zb, 1, 1e-2, 0.9, 0.99, 1e-8, 0.1)
    q, m, v = training.adamw64(p, g, z * 0.0, z * 0.0, 1, 1e-2, 0.9, 0.99, 1e-8, 0.1)
    np.testing.assert_allclose(p1, q, rtol=1e-6, atol=1e-8)
    # codes are within half a step (2^-4 relative, 2^-10 / 448 of the maximum below the normal range)
    for code, mx, x in ((m1, mm, m), (v1, vm, np.sqrt(v))):
        got = carrier.e4m3_decode(code) * training.spread(mx / 448, n)
        assert (np.abs(got - x) <= np.abs(x) * (2.0 ** -4 + 1e-6) + training.spread(mx, n) * 2.0 ** -10 / 448).all()
    assert mm[1] == 0 and vm[1] == 0 and not m1[256:512].any()


def test_nearest_second_moment_stalls_and_stochastic_follows():
    # a block whose largest element is constant while the others' gradients grow threefold: to nearest, v's relative
    # change per step (8 (1 - beta2) = 0.8%) is below half a code, so the root stays; stochastically it follows
    n, beta2 = 256, 0.999
    g = np.full(n, 0.3, np.float32)
    g[0] = 30.0
    p = np.zeros(n, np.float32)
    start = training.adamw_e4m3(p, g, np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(1, np.float32),
                                np.zeros(1, np.float32), 1, 0.0, 0.9, 0.0, 1e-8)
    g2 = g.copy()
    g2[1:] = 0.9
    root = {}
    for seed in (None, 11):
        _, m, v, mm, vm = start
        for t in range(2, 1002):
            _, m, v, mm, vm = training.adamw_e4m3(p, g2, m, v, mm, vm, t, 0.0, 0.9, beta2, 1e-8, seed=seed)
        root[seed] = float(np.mean((carrier.e4m3_decode(v) * vm[0] / 448)[1:]))
    want = np.sqrt(0.09 * beta2 ** 1000 + 0.81 * (1 - beta2 ** 1000))     # 0.73
    assert root[None] < 0.35
    assert abs(root[11] - want) < 0.1 * want


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_gradient_by_differences(residual):
    r = RNG(6)
    h, dy, gain = r.standard_normal((3, 17)), r.standard_normal((3, 17)), r.standard_normal(17)
    ds = r.standard_normal((3, 17)) if residual else None
    loss = lambda h, gain: float(np.sum(dy * training.rmsnorm64(h, gain, 1e-3)[1]) + (np.sum(ds * h) if residual else 0))  # noqa: E731
    dx, dgain = training.rmsnorm_grad64(dy, h, gain, 1e-3, ds)
    for _ in range(5):
        a, b = r.standard_normal((3, 17)), r.standard_normal(17)
        e = 1e-6
        num = (loss(h + e * a, gain + e * b) - loss(h - e * a, gain - e * b)) / (2 * e)
        assert abs(num - float(np.sum(dx * a) + np.sum(dgain * b))) < 1e-7
