"""The stochastic requantisation of 8-bit AdamW states at the edge of its
definition: a value goes up where its fraction of a code's step and the random
16 bits together reach 1, and stays down where they miss it by 2^-22 of a step."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import carrier, rng, training

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [1, 2, 3, 8, 12])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("of", ["m", "v"])
def test_fractions_that_just_reach_or_just_miss_a_step(of, up, steps):
    # without decay the new m is the gradient and the new root its magnitude; element 0 makes the block's factor 1
    n, seed, t = 256, 0x1122334455667788, 3
    j = np.arange(n // 4, dtype=np.uint64)
    ctr = np.stack([j, j * 0, j * 0, j * 0 + np.uint64(t)], 1)
    w = rng.philox4x32_10(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)
    u = ((w & 0xFFFF) if of == "m" else (w >> 16)).astype(np.float64) / 65536
    # on a grid of 2^-9 below 8 steps, of 2^-8 above
    g = (steps + (1 - u - (0 if up else 2.0 ** -22)) * (1 if steps < 8 else 2)) * 2.0 ** -9
    g = g.astype(np.float32)
    g[1::2] *= -1 if of == "m" else 1
    g[0] = 448.0
    p, grad = torch.zeros(n, device="cuda"), torch.from_numpy(g).cuda()
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    mm, vm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    plan = q.qmuon_adamw_plan_create([q.adamw_tensor(p, grad, m, v, n, "f32", mm, vm)], "e4m3")
    q.qmuon_adamw_step_sr(plan, t, 0.0, 0.0, 0.0, 1e-8, seed)
    z, zb = np.zeros(n, np.uint8), np.zeros(1, np.float32)
    _, mc, vc, _, _ = training.adamw_e4m3(np.zeros(n, np.float32), g, z, z, zb, zb, t, 0.0, 0.0, 0.0, 1e-8, seed=seed)
    got, want = (m, mc) if of == "m" else (v, vc)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    to = carrier.e4m3_decode(want)[1:] * 512
    if steps < 8:     # the definition itself, where the fraction is exact
        assert (np.abs(to) == steps + (1 if up else 0)).all()
