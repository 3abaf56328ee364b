"""What a plan uploads is on the device before its creation returns: a step may
follow at once on a stream that nothing orders after the upload."""

import glob
import os
import re

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
import workloads

CSRC = os.path.join(os.path.dirname(os.path.abspath(q.__file__)), "csrc")


def test_every_synchronous_upload_waits():
    # cudaMemcpy from pageable memory may return before the copy to the device is done, and orders itself with the legacy
    # stream alone: host-to-device copies that are not on a caller's stream go through the one helper that waits
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not path.endswith((".cu", ".h")):
            continue
        text = open(path).read()
        for m in re.finditer(r"\bcudaMemcpy(ToSymbol)?\s*\(", text):
            call = text[m.start():text.index(";", m.start())]
            if m.group(1) or "cudaMemcpyHostToDevice" in call:
                found.setdefault(os.path.basename(path), []).append(" ".join(call.split()))
    assert list(found) == ["qm_internal.h"], found
    assert len(found["qm_internal.h"]) == 1
    body = open(os.path.join(CSRC, "qm_internal.h")).read()
    body = body[body.index("upload_and_wait("):]
    assert "cudaStreamSynchronize" in body[:body.index("\n}")]


@pytest.mark.gpu
def test_steps_right_after_creation_on_a_non_blocking_stream():
    # tables of a few hundred KB and more, built and used at once, several times over
    stream = torch.cuda.Stream()
    n = 6000
    gen = torch.Generator("cuda").manual_seed(1)
    flat = {k: torch.randn(n * 64, generator=gen, device="cuda") for k in ("p", "g", "m")}
    flat["v"] = torch.randn(n * 64, generator=gen, device="cuda").square()
    start = {k: t.clone() for k, t in flat.items()}
    part = lambda k: flat[k].view(n, 64).unbind(0)   # noqa: E731
    views = {k: part(k) for k in flat}
    norm, plans = torch.zeros(2, device="cuda"), []
    ws = torch.empty(n * 8 + 256, dtype=torch.uint8, device="cuda")      # at most a double per chunk
    want = None
    for rep in range(5):
        for k in flat:
            flat[k].copy_(start[k])
        torch.cuda.synchronize()
        cp = q.qmuon_clip_plan_create([(g, "f32") for g in views["g"]])
        q.qmuon_grad_clip(cp, 0.5, True, norm, ws, stream=stream)
        ap = q.qmuon_adamw_plan_create([q.adamw_tensor(p, g, m, v, 64, "f32") for p, g, m, v in zip(*(views[k] for k in "pgmv"))])
        q.qmuon_adamw_step(ap, 2, 1e-2, 0.9, 0.99, 1e-8, stream=stream)
        plans += [cp, ap]      # so that no table lies where an earlier one lay
        stream.synchronize()
        got = {k: t.clone() for k, t in flat.items()}
        if want is None:
            # one tensor in the place of all of them
            for k in flat:
                flat[k].copy_(start[k])
            one = q.qmuon_adamw_plan_create([q.adamw_tensor(*(flat[k] for k in "pgmv"), n * 64, "f32")])
            flat["g"].copy_(got["g"])
            q.qmuon_adamw_step(one, 2, 1e-2, 0.9, 0.99, 1e-8)
            torch.cuda.synchronize()
            want = {k: t.clone() for k, t in flat.items()}
            ref = start["g"].double().norm().item()
            assert abs(norm[0].item() - ref) <= 1e-6 * ref
            assert torch.equal(got["g"], start["g"] * norm[1])
        for k in flat:
            assert torch.equal(got[k], want[k]), (rep, k)


@pytest.mark.gpu
def test_a_muon_plan_right_after_creation_on_a_non_blocking_stream():
    stream = torch.cuda.Stream()
    mats = [workloads.Matrix(f"m{i}", 256, 512) for i in range(64)]
    outs = []
    for side in (None, stream):
        state = [workloads.random_state(m, 5 + i, device="cuda") for i, m in enumerate(mats)]
        gen = torch.Generator("cuda").manual_seed(2)
        grads = [torch.randn(m.rows, m.cols, generator=gen, device="cuda").bfloat16() for m in mats]
        weights = [torch.zeros(m.rows, m.cols, device="cuda") for m in mats]
        torch.cuda.synchronize()
        plan = q.qmuon_plan_create([(a, b, g, m.rows, m.cols) for (a, b), g, m in zip(state, grads, mats)])
        ws = torch.empty(q.qmuon_workspace_size(plan, q.QMUON_WS_STEP), dtype=torch.uint8, device="cuda")
        q.qmuon_step_prepare(plan, weights, ws)
        q.qmuon_step(plan, 1, 1, 0.95, 0.02, 0.02, weights, workloads.COEFFS, 5, None, ws, stream=side)
        q.qmuon_sync_status(ws, stream=side)
        outs.append([w.cpu().numpy() for w in weights] + [s[0].cpu().numpy() for s in state])
    for a, b in zip(*outs):
        np.testing.assert_array_equal(a, b)
