"""The gradient norm where single sums are the least exact, and at the ends of
its range.

u = 2^-24.  A thread squares up to 32 elements of a chunk into four running
sums: at most 10 additions of positive terms in one, 2 to join them, fp64 from
there on; halved by the root, with the square's and the norm's own rounding
under 8 u.
"""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _norm(t, name):
    plan = q.qmuon_clip_plan_create([(t, name)])
    ws = torch.empty(q.qmuon_clip_workspace_size(plan), dtype=torch.uint8, device="cuda")
    norm = torch.empty(2, device="cuda")
    q.qmuon_grad_clip(plan, float("inf"), False, norm, ws)
    assert norm[1].item() == 1.0
    return norm[0].item()


@pytest.mark.parametrize("n", [8192, 8191, 3 * 8192 + 2100])
@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("dtype,b", [("f32", 2.0 ** -12 * (1 + 2.0 ** -20)), ("bf16", 2.0 ** -12 * (1 + 2.0 ** -7)),
                                     ("f16", 2.0 ** -12 * (1 + 2.0 ** -10))])
def test_squares_that_all_round_up(dtype, b, off, n):
    # 1 first in every thread's run, then squares a little over half an ulp of 1: each addition to the sum that holds the
    # 1 rounds up by almost u
    x = torch.full((n + off,), b, dtype=DT[dtype], device="cuda")
    t = x[off:]
    for s in range(0, n, 8192):
        t[s:s + 256] = 1.0
    want = np.linalg.norm(t.double().cpu().numpy())
    assert abs(_norm(t, dtype) - want) <= 8 * U * want


@pytest.mark.parametrize("off", [0, 1])
def test_ends_of_the_range(off):
    n = 8192
    x = torch.randn(n + off, generator=torch.Generator("cuda").manual_seed(1), device="cuda")[off:]
    one = torch.full((n + off,), 1.0, device="cuda")[off:]
    for scale in (3e-19 * 2 ** 6, 1e17):      # squares of a normal fp32 and above; sums of 32 that stay finite
        t = torch.empty(n + off, device="cuda")[off:]
        t.copy_(torch.where(x.abs() < 2.0 ** -5, 2.0 ** -5, x) * scale)
        want = np.linalg.norm(t.double().cpu().numpy())
        assert abs(_norm(t, "f32") - want) <= 8 * U * want
    t = torch.empty(n + off, device="cuda")[off:]
    big = t.copy_(one * 3e18)
    assert abs(_norm(big, "f32") - 3e18 * n ** 0.5) <= 1e-6 * 3e18 * n ** 0.5
    # below 1e-19 squares are subnormal: exact to 2^-150 each, sums of them exactly
    tiny = t.copy_(one * 1e-21)
    want = np.linalg.norm(tiny.double().cpu().numpy())
    assert abs(_norm(tiny, "f32") - want) <= want * (0.5 * 2.0 ** -150 / 1e-42 * 1.01 + 8 * U)
    assert _norm(t.copy_(one * 1e-23), "f32") == 0.0       # below 2^-75.5 none is left
