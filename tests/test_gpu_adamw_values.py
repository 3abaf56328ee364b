"""AdamW steps at values that fp32 does not hold, and with gradients that are
not finite."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import training

from test_gpu_adamw import U, _f32_case, _np

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
