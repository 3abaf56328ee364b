"""What the header says of a gated block's calls beside their values: the
workspace of an empty call."""

import pytest
import torch

import memory_reduced_muon_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
def test_an_empty_call_leaves_its_workspace_alone(accumulate):
    """Neither a new workspace's bytes nor a failure that an earlier call recorded are its own to report or to clear."""
    w = torch.ones(5, 16, dtype=torch.bfloat16, device="cuda")
    none, h = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 5, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    forward = q.gated_ffn(none, w, w, h, 0, 16, 5, "bf16")
    grad = q.gated_ffn_grad(h, none, w, w, none, w.clone(), w.clone(), 0, 16, 5, "bf16", accumulate=accumulate)
    q.qmuon_gated_ffn_forward(forward, ws)
    q.qmuon_gated_ffn_backward(grad, ws)
    torch.cuda.synchronize()
    assert bool((ws == 0xFF).all())
    ws.zero_()
    ws[:4].view(torch.int32).fill_(q.QMUON_ERR_TIMEOUT)      # of an earlier call, not yet read
    q.qmuon_gated_ffn_forward(forward, ws)
    q.qmuon_gated_ffn_backward(grad, ws)
    with pytest.raises(q.QmuonError) as e:
        q.qmuon_sync_status(ws)
    assert e.value.status == q.QMUON_ERR_TIMEOUT
    q.qmuon_sync_status(ws)
    # and none is needed
    q.qmuon_gated_ffn_forward(forward, None, ws_bytes=0)
    q.qmuon_gated_ffn_backward(grad, None, ws_bytes=0)
