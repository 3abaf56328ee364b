"""What the header says of a gated block's calls beside their values: the
workspace of an empty call, the order of the sums."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_embedding import Matrix, _np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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


@pytest.mark.parametrize("width,same", [(256, True), (2048, False)])
def test_rows_off_16_bytes_may_change_the_last_bits(width, same):
    """64 x width x 256: the same values in rows that start on 16 bytes and in others.  `same`: both through one kernel, in
    one order.  Otherwise each sum is within its own bound of the exact one, and a fp16 result rounds it once."""
    rows, inner = 64, 256
    gen = torch.Generator("cuda").manual_seed(1)
    x, wg, wu = (torch.randn(n, width, generator=gen, device="cuda").half() * f for n, f in ((rows, 1.0), (inner, width ** -0.5), (inner, width ** -0.5)))
    got = []
    for pad in (0, 8, 3):
        m = [Matrix(t.shape[0], width, pad, torch.float16, 0, t) for t in (x, wg, wu)]
        h, gate, up = (torch.empty(rows, inner, dtype=torch.float16, device="cuda") for _ in range(3))
        call = q.gated_ffn(*(v.t for v in m), h, rows, width, inner, "f16", saved="same", gate=gate, up=up, ld_x=m[0].ld, ld_w_gate=m[1].ld,
                           ld_w_up=m[2].ld)
        ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
        q.qmuon_gated_ffn_forward(call, ws)
        q.qmuon_sync_status(ws)
        got.append((h, gate, up))
    for a, b, c in zip(*got):
        assert torch.equal(a, b)                       # a stride of its own changes nothing
        if same:
            assert torch.equal(a, c)
    X = _np(x)
    for k, w in ((1, wg), (2, wu)):
        e = 2 * width * U * (np.abs(X) @ np.abs(_np(w)).T)
        a, c = _np(got[0][k]), _np(got[2][k])
        # two roundings of values that lie within 2 e of each other
        assert (np.abs(a - c) <= 2 * e + 2.0 ** -11 * (np.abs(a) + np.abs(c)) * (1 + 2.0 ** -10) + 2.0 ** -24).all()
