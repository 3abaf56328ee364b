"""The gated block's backward pass in fp16 with gradients that fp16 can barely
hold: dgate and dup, its operands, must not lose what dh has.

u = 2^-24.  The two are held times a power of two that brings dh's largest
magnitude m to 1/4 or more, so that each is rounded by 2^-11 of itself, or by
2^-25 (half of fp16's smallest number) over that power, 2^-25 m / (1/4) =
2^-23 m.  A product of K terms adds 2 (K + 1) u of the sum of its magnitudes,
as in the tests of the ordinary range; an fp32 result is rounded by u, an fp16
one by 2^-11 or 2^-25."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import activations as act

from test_gpu_embedding import Matrix, _np
from test_gpu_ffn import _err, _kept, _workspace

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F16 = torch.float16


def _call(shape, saved, name, dh, grad_dtype="f32", seed=3):
    """(results, operands in fp64) of one call."""
    rows, width, inner, pad, off = shape
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    x, wg, wu = (Matrix(r, width, pad, F16, off, rnd(r, width) * f) for r, f in ((rows, 1.0), (inner, width ** -0.5), (inner, width ** -0.5)))
    d = Matrix(rows, inner, pad, F16, off, dh)
    kept, lds, E = _kept(rows, inner, pad, off, "f16", saved), {}, np.zeros((rows, inner))
    X, G, W = _np(x.t), _np(wg.t), _np(wu.t)
    if saved == "none":
        gate, up = X @ G.T, X @ W.T
        eg, eu = 2 * width * U * (np.abs(X) @ np.abs(G).T), 2 * width * U * (np.abs(X) @ np.abs(W).T)
    else:
        values, eg, eu = [rnd(rows, inner) for _ in range(2)], E, E
        for k, v in zip(("gate", "up"), values):
            if saved == "same":
                kept[k].t.copy_(v)
            else:
                codes, scale = act.encode(v.cpu().numpy())
                kept[k].t.copy_(torch.from_numpy(codes))
                kept[k + "_scale"].t.copy_(torch.from_numpy(scale))
        if saved == "same":
            gate, up = _np(kept["gate"].t), _np(kept["up"].t)
            lds = dict(ld_gate=kept["gate"].ld, ld_up=kept["up"].ld)
        else:
            gate, up = (act.decode64(kept[k].t.cpu().numpy(), kept[k + "_scale"].t.cpu().numpy()) for k in ("gate", "up"))
    out = {"dx": Matrix(rows, width, pad, F16, off)}
    out["dw_gate"], out["dw_up"] = (Matrix(inner, width, pad, {"f16": F16, "f32": torch.float32}[grad_dtype], off) for _ in range(2))
    call = q.gated_ffn_grad(d.t, x.t, wg.t, wu.t, *(m.t for m in out.values()), rows, width, inner, "f16", act=name, saved=saved,
                            grad_dtype=grad_dtype, ld_dh=d.ld, ld_x=x.ld, ld_w_gate=wg.ld, ld_w_up=wu.ld,
                            **{"ld_" + k: m.ld for k, m in out.items()}, **{k: m.t for k, m in kept.items()}, **lds)
    ws = _workspace(q.qmuon_gated_ffn_backward_workspace_size(call))
    q.qmuon_gated_ffn_backward(call, ws.t)
    q.qmuon_sync_status(ws.t)
    ws.check()
    for m in out.values():
        m.check()
    return {k: m.t for k, m in out.items()}, (X, G, W, gate, up, eg, eu, _np(d.t))


# by elements and by rows of lanes; through the cores' registers, by tiles of 64 and of 128 columns, in splits, straight to
# the results and through partial sums
SHAPES = [(5, 64, 96, 0, 0), (60, 200, 416, 0, 0), (129, 65, 160, 3, 1), (257, 1100, 384, 0, 0), (3001, 64, 2016, 0, 0), (2600, 136, 608, 0, 0),
          (300, 72, 2016, 5, 3)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("saved,name", [("none", "silu"), ("same", "gelu"), ("mxfp8", "gelu_tanh")])
@pytest.mark.parametrize("size", [1e-2, 1e-5, 3e-6])
def test_small_gradients(shape, saved, name, size):
    rows, width, inner = shape[:3]
    gen = torch.Generator("cuda").manual_seed(11)
    dh = torch.randn(rows, inner, generator=gen, device="cuda") * size
    got, (X, G, W, gate, up, eg, eu, DH) = _call(shape, saved, name, dh)
    top = np.abs(DH).max()
    a, slope = act.act64(name, gate)
    e_act = _err(gate) * (np.abs(gate) + 1)
    es, ea = e_act + 0.8 * eg, e_act + 1.13 * eg
    dgate, dup, _ = act.gated_slopes64(DH, gate, up, name)
    # what the arithmetic loses, and the rounding
    off = [e + 2.0 ** -11 * (np.abs(v) + e) + 2.0 ** -23 * top
           for v, e in ((dgate, np.abs(DH) * (np.abs(up) * es + (np.abs(slope) + es) * eu) + 4 * U * np.abs(dgate)),
                        (dup, np.abs(DH) * ea + 4 * U * np.abs(dup)))]
    want = dict(zip(("dx", "dw_gate", "dw_up"), act.gated_products64(dgate, dup, X, G, W)))
    mag = dict(zip(want, act.gated_products64(np.abs(dgate), np.abs(dup), np.abs(X), np.abs(G), np.abs(W))))
    by = dict(zip(want, act.gated_products64(*off, np.abs(X), np.abs(G), np.abs(W))))
    for k, terms in (("dx", 2 * inner), ("dw_gate", rows), ("dw_up", rows)):
        err = 2 * (terms + 1) * U * (mag[k] + by[k]) + by[k]
        bound = err + (2.0 ** -11 * (np.abs(want[k]) + err) + 2.0 ** -25 if k == "dx" else U * (np.abs(want[k]) + err))
        assert (np.abs(_np(got[k]) - want[k]) <= bound).all(), k
        if k != "dx" and rows >= 100:
            # independent roundings: the norm of what is lost, against the norm of what is there.  2^-11 / sqrt 3 of a
            # value each, twice that for what lies below fp16's normal range
            assert np.linalg.norm(_np(got[k]) - want[k]) <= 2.0 ** -10 * np.linalg.norm(want[k]), k


@pytest.mark.parametrize("saved", ["none", "same", "mxfp8"])
@pytest.mark.parametrize("shape", [(60, 200, 416, 0, 0), (257, 1100, 384, 0, 0), (129, 65, 160, 3, 1)], ids=str)
def test_the_scale_leaves_the_bits(shape, saved):
    """dh in powers of two from one size to another: where nothing is lost the results move by the power alone."""
    rows, _, inner = shape[:3]
    gen = torch.Generator("cuda").manual_seed(12)
    dh = torch.randn(rows, inner, generator=gen, device="cuda").half()
    dh[dh.abs() < 2.0 ** -4] = 0.0                          # stays normal in fp16 when divided by 2^10
    base, _ = _call(shape, saved, "silu", dh)
    less, _ = _call(shape, saved, "silu", dh.float() * 2.0 ** -10)
    for k in ("dw_gate", "dw_up"):                          # fp32
        a, b = base[k].double(), less[k].double() * 2.0 ** 10
        # dgate and dup are the same numbers where both are normal in fp16.  Else the one is off by 2^-25 and the other by
        # that over its power: dh below 8 leaves 2^-7 at the end, which 2^5 brings to 1/4, so 2^-25 2^10 / 2^5 at most; |x|
        # is below 6, and fp32 results of one sum are compared
        assert bool(((a - b).abs() <= rows * 6 * (2.0 ** -20 + 2.0 ** -25) + 4 * U * a.abs()).all()), k


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("saved", ["none", "same"])
@pytest.mark.parametrize("shape", [(60, 200, 416, 0, 0), (257, 1100, 384, 0, 0), (129, 65, 161, 3, 1)], ids=str)
def test_values_that_are_not_finite_set_no_scale(shape, saved, bad):
    rows, _, inner = shape[:3]
    gen = torch.Generator("cuda").manual_seed(13)
    dh = torch.randn(rows, inner, generator=gen, device="cuda") * 1e-5
    dh[1, 3] = 0.0
    clean, _ = _call(shape, saved, "silu", dh)
    dh[1, 3] = bad
    got, _ = _call(shape, saved, "silu", dh)
    keep = torch.arange(rows, device="cuda") != 1
    assert torch.equal(got["dx"][keep], clean["dx"][keep]) and not bool(torch.isfinite(got["dx"][1]).any())
    keep = torch.arange(inner, device="cuda") != 3
    for k in ("dw_gate", "dw_up"):
        assert torch.equal(got[k][keep], clean[k][keep]) and not bool(torch.isfinite(got[k][3]).any())


def test_no_gradient_at_all():
    for shape in ((60, 200, 416, 0, 0), (257, 1100, 384, 0, 0)):
        got, _ = _call(shape, "none", "silu", torch.zeros(shape[0], shape[2], device="cuda"), grad_dtype="f16")
        for t in got.values():
            assert bool((t == 0).all())
