"""8-bit AdamW states of blocks whose elements differ by many orders: an element
whose root lies far below its block's maximum must not divide its momentum by
eps alone.

AdamW itself moves an element by at most K lr, K = (1 - b1) / sqrt((1 - b2)
(1 - b1^2 / b2)) (Cauchy-Schwarz over the gradients; the bias corrections only
lower it).  In 8 bits the momentum is off by at most half a code, 2^-4, per step,
which is carried on with weight b1: 2^-4 / (1 - b1) = 0.63 in all; a root is too
small by at most half a code.  1.63 / (1 - 2^-4) < 2: steps of at most 2 K lr.
"""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import carrier, training

B1, EPS, LR = 0.9, 1e-8, 1.0


def _limit(b2):
    return 2 * (1 - B1) / np.sqrt((1 - b2) * (1 - B1 ** 2 / b2)) * LR


def _gradients(kind, n=256):
    """Gradients of the steps of one block."""
    if kind == "spike":             # one element long ago, another one much later
        g = [np.zeros(n, np.float32) for _ in range(72)]
        g[0][0], g[49][1] = 10.0, 1e-5
    elif kind == "first":           # all at the first step, 1e6 apart, then none
        g = [np.full(n, 1e-6, np.float32), np.zeros(n, np.float32), np.zeros(n, np.float32)]
        g[0][0] = 1.0
    else:                           # an element falls silent, the others go on at 1e-7 of it, then none
        g = [np.full(n, 1e-3, np.float32) for _ in range(60)]
        for x in g:
            x[0] = 0.0
        g[0][:], g[-1][:] = 0.0, 0.0
        g[0][0] = 1e4
    return g


KINDS = ["spike", "first", "silent"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("b2", [0.99, 0.999])
@pytest.mark.parametrize("seed", [None, 5, 6])
def test_no_step_runs_away(kind, b2, seed):
    n = 256
    p, m, v = np.zeros(n, np.float32), np.zeros(n, np.uint8), np.zeros(n, np.uint8)
    mm = vm = np.zeros(1, np.float32)
    for t, g in enumerate(_gradients(kind), 1):
        p1, m, v, mm, vm = training.adamw_e4m3(p, g, m, v, mm, vm, t, LR, B1, b2, EPS, seed=seed)
        assert np.abs(p1 - p).max() <= _limit(b2), t
        p = p1


@pytest.mark.parametrize("seed", [None, 3])
def test_a_positive_root_keeps_a_code(seed):
    # roots from 1e-9 of the block's to 1: code 1 at least, code 0 for zero alone
    g = np.float32(10.0) ** np.linspace(-9, 0, 256, dtype=np.float32)
    g[::7] = 0.0
    z, zb = np.zeros(256, np.uint8), np.zeros(1, np.float32)
    _, _, v, _, vm = training.adamw_e4m3(np.zeros(256, np.float32), g, z, z, zb, zb, 1, LR, B1, 0.99, EPS, seed=seed)
    np.testing.assert_array_equal(v == 0, g == 0)
    got = carrier.e4m3_decode(v) * vm[0] / 448
    root = 0.1 * g.astype(np.float64)
    # a code's step: 2^-3 of a value, or 2^-9 / 448 of the maximum (stochastically up to a whole one)
    assert (np.abs(got - root) <= np.maximum(root * 2.0 ** -3, 2.0 ** -9 / 448 * vm[0]) * (1 + 1e-6)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("grad", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("sizes", [[256, 2000, 5], [256 * 8 * 3 * 400]], ids=["one block per warp", "three"])
def test_kernel_keeps_codes_of_small_roots(sizes, sr, grad):
    # bit for bit the definition, on blocks whose gradients and states spread over nine orders (f16: over its subnormals)
    from test_gpu_adamw import DT, _check_e4m3, _e4m3_case, _host
    ts, guards, plan = _e4m3_case(sizes, grad, None, 0, 17)
    gen = torch.Generator("cuda").manual_seed(18)
    for d in ts:
        n = d["n"]
        e = torch.rand(n, generator=gen, device="cuda") * -9
        e[::256] = 1.0
        d["grad"].copy_(torch.where(torch.rand(n, generator=gen, device="cuda") < 0.2, 0.0, 10.0 ** e).to(DT[grad]))
        old = torch.rand(n, generator=gen, device="cuda")
        d["v"][old < 0.5] = 0
        d["m"][old < 0.5] = 0
    for t in (4, 5):
        host = _host(ts)
        if sr:
            q.qmuon_adamw_step_sr(plan, t, 1e-2, B1, 0.99, EPS, 21)
        else:
            q.qmuon_adamw_step(plan, t, 1e-2, B1, 0.99, EPS)
        torch.cuda.synchronize()
        _check_e4m3(ts, host, t, 1e-2, B1, 0.99, EPS, 1.0, 21 if sr else None)
    small = [int((d["v"] == 1).sum()) for d in ts]
    assert small[0] > 0
    for g in guards:
        g.check()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("b2", [0.99, 0.999])
@pytest.mark.parametrize("sr", [False, True])
def test_no_step_of_the_kernel_runs_away(kind, b2, sr):
    n = 256
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    mm, vm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    plan = q.qmuon_adamw_plan_create([q.adamw_tensor(p, g, m, v, n, "f32", mm, vm)], "e4m3")
    for t, x in enumerate(_gradients(kind), 1):
        g.copy_(torch.from_numpy(x))
        before = p.clone()
        if sr:
            q.qmuon_adamw_step_sr(plan, t, LR, B1, b2, EPS, 5)
        else:
            q.qmuon_adamw_step(plan, t, LR, B1, b2, EPS)
        assert float((p - before).abs().max()) <= _limit(b2), t
