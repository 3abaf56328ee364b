"""AdamW steps at values that fp32 does not hold, with gradients that are not
finite, and of dense 8-bit states in the kernels for many blocks."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_adamw import _f32_case

pytestmark = pytest.mark.gpu


def test_rates_that_fp32_does_not_hold_are_refused():
    ts, _, plan = _f32_case([300], "bf16", "bf16", 0, 5)
    before = {k: ts[0][k].clone() for k in ("param", "m", "v", "copy")}
    for lr, eps in ((1e39, 1e-8), (-1e300, 1e-8), (1e-3, 1e39)):
        with pytest.raises(q.QmuonError) as e:
            q.qmuon_adamw_step(plan, 1, lr, 0.9, 0.99, eps)
        assert e.value.status == q.QMUON_ERR_INVALID_ARGUMENT
    torch.cuda.synchronize()
    for k, t in before.items():
        assert torch.equal(t, ts[0][k])
    q.qmuon_adamw_step(plan, 1, 3e37, 0.9, 0.99, 3e38)      # lr / (1 - beta1) and eps are within its range
    assert bool(torch.isfinite(ts[0]["param"]).all())


def test_the_smallest_eps_is_taken():
    ts, _, plan = _f32_case([300], "bf16", None, 0, 5)
    q.qmuon_adamw_step(plan, 1, 1e-3, 0.9, 0.99, 1.17549435e-38)      # rounds to 2^-126
    assert bool(torch.isfinite(ts[0]["param"]).all())


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("grad", ["bf16", "f16", "f32"])
def test_f32_states_keep_what_is_not_finite_to_its_element(grad, off):
    n, bad = 5000, {3: float("nan"), 2047: float("inf"), 2500: -float("inf"), 4999: float("nan")}
    runs = []
    for put in (False, True):
        ts, guards, plan = _f32_case([n], grad, "bf16", off, 23)
        clean = ts[0]["grad"].clone()
        if put:
            for i, x in bad.items():
                ts[0]["grad"][i] = x
        q.qmuon_adamw_step(plan, 1, 1e-2, 0.9, 0.99, 1e-8)
        ts[0]["grad"].copy_(clean)
        q.qmuon_adamw_step(plan, 2, 1e-2, 0.9, 0.99, 1e-8)
        torch.cuda.synchronize()
        for g in guards:
            g.check()
        runs.append({k: ts[0][k].float().cpu().numpy() for k in ("param", "m", "v", "copy")})
    where = np.zeros(n, bool)
    where[list(bad)] = True
    for k, got in runs[1].items():
        np.testing.assert_array_equal(got[~where], runs[0][k][~where])
        assert not np.isfinite(got[where]).any(), k
    assert np.isnan(runs[1]["param"][where]).all()       # infinity over infinity too


@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("grad,copy", [("bf16", None), ("bf16", "f16"), ("f16", "bf16"), ("f32", None), ("f32", "bf16")])
def test_dense_8_bit_states_by_three_blocks_per_warp(grad, copy, sr):
    # enough blocks for the kernels of three blocks per warp, the last chunk and the last block not whole; every element's
    # codes, maxima and parameter against the definition, every copy against its parameter
    from test_gpu_adamw import DT, _check_e4m3, _e4m3_case, _host
    ts, guards, plan = _e4m3_case([3 * 8 * 256 * 310 + 5 * 256 + 77, 3 * 8 * 256 + 1], grad, copy, 0, 31)
    host = _host(ts)
    scale = torch.full((1,), 0.37, device="cuda")
    if sr:
        q.qmuon_adamw_step_sr(plan, 5, 1e-2, 0.9, 0.99, 1e-8, 99, scale)
    else:
        q.qmuon_adamw_step(plan, 5, 1e-2, 0.9, 0.99, 1e-8, scale)
    torch.cuda.synchronize()
    _check_e4m3(ts, host, 5, 1e-2, 0.9, 0.99, 1e-8, float(np.float32(0.37)), 99 if sr else None)
    for d in ts:
        assert torch.equal(d["copy"], d["param"].to(DT[copy]) if copy else torch.zeros_like(d["copy"]))
    for g in guards:
        g.check()
