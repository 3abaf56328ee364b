"""The gated block's gradients over the longest sums that the header allows.
The tensor-core kernel's waits are bounded, and its epilogue waits for a whole
unit of work: such a sum is taken in pieces, which the workspace has room for."""

import ctypes as C
import os

import pytest
import torch

import memory_reduced_muon_gb300 as q

FAKE = 0x7F0000000000   # never dereferenced


def _size(rows, width, inner, dx=True, dw=True):
    if not os.path.exists(q.LIB_PATH):
        from memory_reduced_muon_gb300 import build
        build.build()
    p = [FAKE] * 13
    p[2] = None                                        # x_scale
    if not dx:
        p[9] = None
    if not dw:
        p[10] = p[11] = None
    p[12] = None                                       # h
    lds = [inner, width, width, width, inner, inner, width, width, width, inner]
    c = q.qmuon_gated_ffn_grad(*p, rows, width, inner, *lds, q.QMUON_ACT_SILU, q.QMUON_BF16, q.QMUON_SAVE_SAME, q.QMUON_BF16, 0, 0)
    return q.lib().qmuon_gated_ffn_backward_workspace_size(C.byref(c))


def test_long_sums_have_room_for_their_pieces():
    # dx over 2 2^28 columns is 2^23 blocks of K, of 512 cycles of the tensor cores each at least: 4.3e9 where a wait gives up
    # after 4.0e9.  In pieces of 2^20 blocks: 8 of 1 x 8 fp32
    inner = 1 << 28
    assert _size(1, 8, inner) - _size(1, 8, inner, dx=False) == 8 * 8 * 4
    assert _size(1, 8, 1 << 25) == _size(1, 8, 1 << 25, dx=False)          # one piece, straight to the result
    # the weights' gradients over 2^28 rows, 2^22 blocks: 4 pieces of two 64 x 64 (in pieces that few tiles ask for, 8 and
    # more, whatever the length)
    rows = 1 << 28
    assert _size(rows, 64, 64) - _size(rows, 64, 64, dw=False) >= 2 * 4 * 64 * 64 * 4


def test_long_projections_have_room_for_their_pieces():
    # 16 x 8 tiles of 256 x 128 and more are enough for all CTA pairs (76 here); K of 2^20 + 1 blocks
    rows, inner, width = 4032, 1000, (1 << 26) + 64
    c = q.qmuon_gated_ffn(*[FAKE] * 4, *[None] * 4, rows, width, inner, width, width, width, inner, inner, inner, q.QMUON_ACT_SILU,
                          q.QMUON_BF16, q.QMUON_SAVE_NONE, 0)
    assert q.lib().qmuon_gated_ffn_workspace_size(C.byref(c)) == 256 + 2 * 2 * rows * inner * 4
    c.width = c.ld_x = c.ld_w_gate = c.ld_w_up = 1 << 26
    assert q.lib().qmuon_gated_ffn_workspace_size(C.byref(c)) == 256


@pytest.mark.gpu
def test_longest_sum():
    """dx of one row over 2^28 columns, beside weights' gradients of as many tiles: whole numbers, whose sums are exact."""
    rows, width, inner = 1, 8, 1 << 28
    gen = torch.Generator("cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda", dtype=torch.int8).bfloat16()   # noqa: E731
    x, w, dh = whole(rows, width), whole(inner, width), whole(rows, inner)
    gate, up = torch.zeros(rows, inner, dtype=torch.bfloat16, device="cuda"), torch.full((rows, inner), 2.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((rows, width), 9.0, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = torch.full_like(w, 9.0), torch.full_like(w, 9.0)
    # silu(0) = 0 and its slope 1/2: dgate = dh, dup = 0
    call = q.gated_ffn_grad(dh, x, w, w, dx, dwg, dwu, rows, width, inner, "bf16", saved="same", gate=gate, up=up)
    ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_backward(call, ws)
    q.qmuon_sync_status(ws)
    want = torch.zeros(width, dtype=torch.float64, device="cuda")
    for i in range(0, inner, 1 << 24):
        part = slice(i, i + (1 << 24))
        want += (dh[0, part, None].float() * w[part].float()).sum(0, dtype=torch.float64)
        assert torch.equal(dwg[part], dh[0, part, None] * x) and not bool(dwu[part].any())
    assert torch.equal(dx[0], want.bfloat16())
