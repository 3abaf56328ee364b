"""The embedding, the checkpoints and the gated block on arrays of more than
2^31 elements: samples from their ends and middles against fp64.  Bounds as in
the files of the small sizes."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import activations as act

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, U8 = torch.bfloat16, torch.uint8


def _np(t):
    return t.detach().cpu().double().numpy()


def test_embedding_of_a_large_table():
    vocab, cols, n = 530000, 4096, 3000               # 2,170,880,000 elements
    gen = torch.Generator("cuda").manual_seed(1)
    table = torch.empty(vocab, cols, dtype=BF16, device="cuda")
    for i in range(0, vocab, 53000):
        table[i:i + 53000] = torch.randn(53000, cols, generator=gen, device="cuda", dtype=BF16)
    tokens = torch.cat([torch.tensor([0, vocab - 1, vocab - 1, vocab, 524288, 524287], device="cuda"),
                        torch.randint(vocab - 2000, vocab, (n - 6,), generator=gen, device="cuda")])
    out = torch.empty(n, cols, dtype=BF16, device="cuda")
    q.qmuon_embedding_forward(table, tokens, out, n, vocab, cols, "bf16")
    want = torch.where((tokens < vocab)[:, None], table[tokens.clamp(max=vocab - 1)], torch.zeros((), dtype=BF16, device="cuda"))
    assert torch.equal(out, want)
    # the gradient over the table's memory
    dout = torch.randn(n, cols, generator=gen, device="cuda", dtype=BF16)
    ws = torch.empty(q.qmuon_embedding_workspace_size(n, vocab, cols), dtype=U8, device="cuda")
    q.qmuon_embedding_backward(dout, tokens, table, n, vocab, cols, "bf16", ws)
    there = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    there[tokens[tokens < vocab]] = True
    for i in range(0, vocab, 53000):
        part = table[i:i + 53000]
        assert bool((part[~there[i:i + 53000]] == 0).all())
    grad, mag, count = act.embedding_grad64(_np(dout[:, :64]), np.where(_np(tokens) < vocab, _np(tokens), -1).astype(np.int64), vocab)
    rows = np.flatnonzero(count)
    got = _np(table[torch.from_numpy(rows).cuda(), :64])
    bound = (count[rows, None] + 2) * U * mag[rows] + 2.0 ** -8 * np.abs(grad[rows]) + 1e-40
    assert (np.abs(got - grad[rows]) <= bound).all()


def test_checkpoint_of_a_large_activation():
    rows, cols = 67000, 32768                         # 2,195,456,000 elements
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    for i in range(0, rows, 6700):
        x[i:i + 6700] = torch.randn(6700, cols, generator=gen, device="cuda", dtype=BF16)
    pay, sc = torch.empty(rows, cols, dtype=U8, device="cuda"), torch.empty(rows, cols // 32, dtype=U8, device="cuda")
    q.qmuon_mxfp8_encode(x, pay, sc, rows, cols, "bf16")
    at = [0, 1, 33333, 65535, 65536, rows - 2, rows - 1]
    payload, scale = act.encode(x[at].float().cpu().numpy())
    np.testing.assert_array_equal(pay[at].cpu().numpy(), payload)
    np.testing.assert_array_equal(sc[at].cpu().numpy(), scale)
    x.zero_()
    q.qmuon_mxfp8_decode(pay, sc, x, rows, cols, "bf16")
    np.testing.assert_array_equal(_np(x[at]), act.decode64(payload, scale))


def test_gated_block_of_many_rows():
    rows, width, inner = 150001, 64, 14336            # 2,150,414,336 elements of h
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(rows, width, generator=gen, device="cuda", dtype=BF16)
    w = [(torch.randn(inner, width, generator=gen, device="cuda") / 8).to(BF16) for _ in range(2)]
    h = torch.empty(rows, inner, dtype=BF16, device="cuda")
    kept = dict(gate=torch.empty(rows, inner, dtype=U8, device="cuda"), up=torch.empty(rows, inner, dtype=U8, device="cuda"),
                gate_scale=torch.empty(rows, inner // 32, dtype=U8, device="cuda"),
                up_scale=torch.empty(rows, inner // 32, dtype=U8, device="cuda"))
    call = q.gated_ffn(x, *w, h, rows, width, inner, "bf16", saved="mxfp8", **kept)
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=U8, device="cuda")
    q.qmuon_gated_ffn_forward(call, ws)
    q.qmuon_sync_status(ws)
    at = [0, 255, 256, 75000, 149796, 149797, rows - 2, rows - 1]      # around element 2^31 too
    X, G, W = _np(x), _np(w[0]), _np(w[1])
    want, gate, up = act.gated_ffn64(X[at], G, W, "silu")
    eg, eu = (2 * width * U * (np.abs(X[at]) @ np.abs(m).T) for m in (G, W))
    e_act = (16 + 4 * (np.abs(gate) + gate * gate)) * 2 * U * (np.abs(gate) + 1)
    err = 1.13 * eg * (np.abs(up) + eu) + np.abs(act.act64("silu", gate)[0]) * eu + e_act * np.abs(up)
    assert (np.abs(_np(h[at]) - want) <= err + 2.0 ** -8 * (np.abs(want) + err)).all()
    g8, u8 = (act.decode64(kept[k][at].cpu().numpy(), kept[k + "_scale"][at].cpu().numpy()) for k in ("gate", "up"))
    for got, v, e in ((g8, gate, eg), (u8, up, eu)):
        unit = np.repeat(2.0 ** np.ceil(np.log2(np.abs(v.reshape(len(at), -1, 32)).max(2) / 448) + 1e-6), 32, 1)
        assert (np.abs(got - v) <= np.maximum(2.0 ** -4 * (np.abs(v) + e), 2.0 ** -10 * unit) + e).all()
    # backward from the checkpoints; dh takes h's memory, h again other memory
    dh, again = h, torch.empty(rows, inner, dtype=BF16, device="cuda")
    for i in range(0, rows, 30000):
        dh[i:i + 30000] = torch.randn(min(30000, rows - i), inner, generator=gen, device="cuda", dtype=BF16) / 64
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w[0]), torch.empty_like(w[1])
    call = q.gated_ffn_grad(dh, x, *w, dx, dwg, dwu, rows, width, inner, "bf16", saved="mxfp8", h=again, **kept)
    ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=U8, device="cuda")
    q.qmuon_gated_ffn_backward(call, ws)
    q.qmuon_sync_status(ws)
    dgate, dup, h64 = act.gated_slopes64(_np(dh[at]), g8, u8, "silu")
    assert (np.abs(_np(again[at]) - h64) <= 2.0 ** -8 * 1.001 * np.abs(h64) + e_act * np.abs(u8) + 1e-30).all()
    # dgate and dup are off by a rounding (2^-8 at most); 2 inner additions
    dx64 = dgate @ G + dup @ W
    mag = np.abs(dgate) @ np.abs(G) + np.abs(dup) @ np.abs(W)
    rms = np.sqrt((dgate ** 2) @ (G ** 2) + (dup ** 2) @ (W ** 2))
    # independent roundings of standard deviation below 2^-8 / sqrt 3 each: 7 of them
    bound = 7 * 2.0 ** -8 / 3 ** 0.5 * rms + (4 * inner * U + 2.0 ** -18) * mag + 2.0 ** -8 * np.abs(dx64)
    assert (np.abs(_np(dx[at]) - dx64) <= bound).all()
    # columns of the weights' gradients, over all rows
    cols = [0, 127, 128, 7000, inner - 1]
    unit = lambda k: torch.exp2(kept[k + "_scale"][:, [c // 32 for c in cols]].double() - 127)   # noqa: E731
    gc, uc = (kept[k][:, cols].view(torch.float8_e4m3fn).double() * unit(k) for k in ("gate", "up"))
    s = torch.sigmoid(gc)
    dc = dh[:, cols].double()
    for got, d in ((dwg, dc * uc * (s + gc * s * (1 - s))), (dwu, dc * gc * s)):
        want, mag = d.T @ x.double(), d.abs().T @ x.double().abs()
        rms = ((d ** 2).T @ (x.double() ** 2)).sqrt()
        bound = 7 * 2.0 ** -8 / 3 ** 0.5 * rms + (2 * rows * U + 2.0 ** -18) * mag + 2.0 ** -8 * want.abs()
        assert bool(((got[cols].double() - want).abs() <= bound).all())
