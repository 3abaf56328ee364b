"""The gated feed-forward block on the GPU, forward and backward, against fp64:
from one row to many, odd sizes, strides and starts, everything that a forward
pass can keep, guard bytes around what is written, NaN in what is not to be
read.

ut is the stored type's unit roundoff, u = 2^-24.  A product of K terms is
summed in fp32 with at most K additions, each off by 2 u of a magnitude that
sum |a| |b| bounds (tensor cores may cut where fp32 would round): E = 2 K u
sum |a| |b|.  The activations' relative error: the exponential's argument z has
two or three roundings, so exp(z) is off by (4 + 2 |z|) ulp, with |z| at most
g^2 + |g| for these |g|; the rest of the formula, and erfc, add 16 ulp (an ulp
being 2 u): A(g) = (16 + 4 (|g| + g^2)) 2 u of magnitudes that |g| + 1 bounds.
dgate and dup are compared as what the header says, rounded to the type: where
an error within the bound could round to another value, that difference times
the other operand is allowed."""

import itertools

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import activations as act

from gpu_util import Guarded
from test_gpu_embedding import DT, TINY, U, UT, Matrix, _np

pytestmark = pytest.mark.gpu

# rows, width, inner, pad, off: every edge of the tiles of 256 x 128, of the 64 columns of a block of K, splits of K and none
# (of the gradients' products, that is: the projections of all of these are small enough for the cores' registers; those on
# the tensor cores are tested at LARGE, and by their tiles in test_gpu_ffn_tiles.py)
SHAPES = [(1, 64, 128, 0, 0), (1, 1, 1, 0, 0), (2, 8, 31, 0, 0), (3, 257, 33, 3, 1), (127, 63, 129, 0, 0), (128, 64, 127, 8, 0),
          (129, 65, 130, 0, 8), (200, 1000, 96, 16, 0), (256, 128, 256, 0, 0), (257, 200, 384, 0, 0), (300, 72, 1001, 5, 3),
          (1, 4096, 640, 0, 0), (17, 1024, 64, 0, 0), (513, 40, 520, 0, 0)]
# large enough for the tensor-core kernel forward (the smaller ones above go through the cores' registers there)
LARGE = [(257, 1100, 384, 0, 0), (129, 1001, 301, 3, 1), (300, 72, 2001, 5, 3), (1000, 520, 202, 0, 0), (4097, 72, 33, 0, 0), (4100, 1, 1, 0, 0),
         (260, 2056, 200, 8, 8)]
ACTS = ["silu", "gelu", "gelu_tanh"]


def _err(g):
    return (16 + 4 * (np.abs(g) + g * g)) * 2 * U


def _round(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).double().numpy()


def _operands(rows, width, inner, pad, off, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    x = Matrix(rows, width, pad, DT[dtype], off, rnd(rows, width))
    ws = [Matrix(inner, width, pad, DT[dtype], off, rnd(inner, width) * 1.5 * width ** -0.5) for _ in range(2)]
    for m in (x, *ws):
        m.rows[:, width:] = float("nan")      # behind the rows, and before the first: never read into a result
        m.g.t[:off] = float("nan")
    return x, ws[0], ws[1], gen


def _workspace(size):
    ws = Guarded((size,), torch.uint8)
    ws.t.fill_(0xFF)                           # NaN everywhere
    return ws


def _kept(rows, inner, pad, off, dtype, saved):
    if saved == "same":
        return {k: Matrix(rows, inner, pad, DT[dtype], off) for k in ("gate", "up")}
    if saved == "mxfp8":
        return {**{k: Matrix(rows, inner, 0, torch.uint8) for k in ("gate", "up")},
                **{k: Matrix(rows, inner // 32, 0, torch.uint8) for k in ("gate_scale", "up_scale")}}
    return {}


def _forward(shape, dtype, name, saved, seed=1):
    rows, width, inner, pad, off = shape
    x, wg, wu, _ = _operands(*shape, dtype, seed)
    h, kept = Matrix(rows, inner, pad, DT[dtype], off), _kept(rows, inner, pad, off, dtype, saved)
    lds = dict(ld_gate=kept["gate"].ld, ld_up=kept["up"].ld) if saved == "same" else {}
    call = q.gated_ffn(x.t, wg.t, wu.t, h.t, rows, width, inner, dtype, act=name, saved=saved, ld_x=x.ld, ld_w_gate=wg.ld,
                       ld_w_up=wu.ld, ld_h=h.ld, **{k: m.t for k, m in kept.items()}, **lds)
    ws = _workspace(q.qmuon_gated_ffn_workspace_size(call))
    q.qmuon_gated_ffn_forward(call, ws.t)
    q.qmuon_sync_status(ws.t)
    ws.check()
    for m in (h, *kept.values()):
        m.check()
    return x, wg, wu, h, kept


def _projections(x, wg, wu):
    """gate, up and the bounds on their errors."""
    X, G, W = _np(x.t), _np(wg.t), _np(wu.t)
    k = X.shape[1]
    return X @ G.T, X @ W.T, 2 * k * U * (np.abs(X) @ np.abs(G).T), 2 * k * U * (np.abs(X) @ np.abs(W).T)


def _check_forward(shape, dtype, name, saved):
    x, wg, wu, h, kept = _forward(shape, dtype, name, saved)
    gate, up, eg, eu = _projections(x, wg, wu)
    a, _ = act.act64(name, gate)
    want = a * up
    # |act'| is below 1.13
    err = 1.13 * eg * (np.abs(up) + eu) + np.abs(a) * eu + _err(gate) * (np.abs(gate) + 1) * np.abs(up)
    assert (np.abs(_np(h.t) - want) <= err + UT[dtype] * (np.abs(want) + err) + TINY[dtype]).all()
    if saved == "same":
        for m, v, e in ((kept["gate"], gate, eg), (kept["up"], up, eu)):
            assert (np.abs(_np(m.t) - v) <= e + UT[dtype] * (np.abs(v) + e) + TINY[dtype]).all()
    if saved == "mxfp8":
        for k, v, e in (("gate", gate, eg), ("up", up, eu)):
            payload, scale = kept[k].t.cpu().numpy(), kept[k + "_scale"].t.cpu().numpy()
            unit = 2.0 ** (scale.astype(np.float64) - 127)
            top = np.abs(v).reshape(v.shape[0], -1, 32).max(2)
            slack = e.reshape(v.shape[0], -1, 32).max(2)
            assert (top - slack <= 448 * unit).all() and (top + slack > 224 * unit).all()
            half = np.maximum(2.0 ** -4 * (np.abs(v) + e), 2.0 ** -10 * np.repeat(unit, 32, 1))
            assert (np.abs(act.decode64(payload, scale) - v) <= half + e).all()


@pytest.mark.parametrize("shape", SHAPES + LARGE, ids=str)
@pytest.mark.parametrize("dtype,name", list(itertools.product(["bf16", "f16"], ACTS)))
@pytest.mark.parametrize("saved", ["none", "same"])
def test_forward(shape, dtype, name, saved):
    _check_forward(shape, dtype, name, saved)


@pytest.mark.parametrize("shape", [(1, 64, 128, 0, 0), (2, 8, 32, 0, 0), (129, 65, 160, 0, 8), (300, 72, 992, 5, 3), (1, 2048, 64, 0, 0),
                                   (257, 200, 384, 0, 0), (257, 1100, 384, 0, 0), (300, 72, 2016, 5, 3), (4097, 72, 32, 1, 0)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_keeps_8_bits(shape, dtype):
    _check_forward(shape, dtype, "silu", "mxfp8")


def test_forward_of_many_tiles():
    """More tiles than CTA pairs, K long enough to go round the shared-memory ring."""
    for shape in ((1000, 1100, 3000, 0, 0), (2600, 264, 1500, 0, 0)):
        _check_forward(shape, "bf16", "silu", "none")


def _backward(shape, dtype, name, saved, x_mxfp8=False, grad_dtype=None, accumulate=False, again=True, dx=True, dw=True, seed=2):
    """Runs one call, checks all that it writes, and returns it."""
    rows, width, inner, pad, off = shape
    grad_dtype = grad_dtype or dtype
    x, wg, wu, gen = _operands(*shape, dtype, seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    dh = Matrix(rows, inner, pad, DT[dtype], off, rnd(rows, inner))
    dh.rows[:, inner:] = float("nan")
    X, x_arg, extra = _np(x.t), x.t, dict(ld_x=x.ld)
    if x_mxfp8:
        codes, scale = act.encode(X.astype(np.float32))
        X, x_arg, extra = act.decode64(codes, scale), torch.from_numpy(codes).cuda(), dict(x_scale=torch.from_numpy(scale).cuda())
    G, W, DH = _np(wg.t), _np(wu.t), _np(dh.t)
    kept, lds = {}, {}
    if saved == "none":
        gate, up = X @ G.T, X @ W.T
        eg, eu = 2 * width * U * (np.abs(X) @ np.abs(G).T), 2 * width * U * (np.abs(X) @ np.abs(W).T)
    else:
        values = [rnd(rows, inner) * 2 for _ in range(2)]
        kept = _kept(rows, inner, pad, off, dtype, saved)
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
        eg = eu = np.zeros_like(gate)
    out = {}
    if dx:
        out["dx"] = Matrix(rows, width, pad, DT[dtype], off)
    if dw:
        out["dw_gate"], out["dw_up"] = (Matrix(inner, width, pad, DT[grad_dtype], off, rnd(inner, width)) for _ in range(2))
    if again:
        out["h"] = Matrix(rows, inner, pad, DT[dtype], off)
    before = {k: _np(m.t) for k, m in out.items()}
    call = q.gated_ffn_grad(dh.t, x_arg, wg.t, wu.t, *(out[k].t if k in out else None for k in ("dx", "dw_gate", "dw_up")), rows, width,
                            inner, dtype, act=name, saved=saved, h=out["h"].t if again else None, grad_dtype=grad_dtype,
                            accumulate=accumulate, ld_dh=dh.ld, ld_w_gate=wg.ld, ld_w_up=wu.ld,
                            **{"ld_" + k: m.ld for k, m in out.items()}, **{k: m.t for k, m in kept.items()}, **lds, **extra)
    ws = _workspace(q.qmuon_gated_ffn_backward_workspace_size(call))
    q.qmuon_gated_ffn_backward(call, ws.t)
    q.qmuon_sync_status(ws.t)
    ws.check()
    for m in out.values():
        m.check()

    ut = UT[dtype]
    a, slope = act.act64(name, gate)
    e_act = _err(gate) * (np.abs(gate) + 1)
    # |act'| is below 1.13, |act''| below 0.8
    es, ea = e_act + 0.8 * eg, e_act + 1.13 * eg
    if again:
        err = ea * (np.abs(up) + eu) + np.abs(a) * eu
        assert (np.abs(_np(out["h"].t) - a * up) <= err + ut * (np.abs(a * up) + err) + TINY[dtype]).all()
    dgate, dup, _ = act.gated_slopes64(DH, gate, up, name)
    e1 = np.abs(DH) * (np.abs(up) * es + (np.abs(slope) + es) * eu) + 4 * U * np.abs(dgate)
    e2 = np.abs(DH) * ea + 4 * U * np.abs(dup)
    rounded, slack = [], []
    for v, e in ((dgate, e1), (dup, e2)):
        r = _round(v, dtype)
        rounded.append(r)
        slack.append(np.maximum(np.abs(_round(v + e, dtype) - r), np.abs(_round(v - e, dtype) - r)))
    want = dict(zip(("dx", "dw_gate", "dw_up"), act.gated_products64(*rounded, X, G, W)))
    mag = dict(zip(want, act.gated_products64(np.abs(rounded[0]), np.abs(rounded[1]), np.abs(X), np.abs(G), np.abs(W))))
    off_by = dict(zip(want, act.gated_products64(*slack, np.abs(X), np.abs(G), np.abs(W))))
    terms = {"dx": 2 * inner, "dw_gate": rows, "dw_up": rows}
    for k in want:
        if k not in out:
            continue
        w, t = want[k], (dtype if k == "dx" else grad_dtype)
        err = 2 * (terms[k] + 1) * U * (mag[k] + off_by[k]) + off_by[k]
        if accumulate and k != "dx":
            w = w + before[k]
            err = err + 2 * U * np.abs(w)
        got = _np(out[k].t)
        assert (np.abs(got - w) <= err + UT[t] * (np.abs(w) + err) + TINY[t]).all(), k
    return {k: m.t for k, m in out.items()}


@pytest.mark.parametrize("shape", SHAPES + LARGE, ids=str)
@pytest.mark.parametrize("dtype,name,saved", [("bf16", "silu", "none"), ("f16", "gelu", "none"), ("bf16", "gelu_tanh", "same"),
                                              ("f16", "silu", "same"), ("bf16", "gelu", "same"), ("f16", "gelu_tanh", "none")])
def test_backward(shape, dtype, name, saved):
    _backward(shape, dtype, name, saved)


@pytest.mark.parametrize("shape", [(1, 64, 128, 0, 0), (2, 32, 32, 0, 0), (129, 64, 160, 0, 8), (300, 96, 992, 5, 3), (1, 2048, 64, 0, 0),
                                   (257, 224, 384, 0, 0), (1100, 32, 64, 0, 0), (300, 1024, 384, 0, 0), (300, 64, 2016, 5, 3)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("saved,x_mxfp8", [("mxfp8", True), ("mxfp8", False), ("none", True), ("same", True)])
def test_backward_from_8_bits(shape, dtype, saved, x_mxfp8):
    _backward(shape, dtype, "silu", saved, x_mxfp8)


@pytest.mark.parametrize("shape", [(300, 72, 1001, 5, 3), (257, 200, 384, 0, 0), (1, 64, 128, 0, 0), (5000, 64, 64, 0, 0)], ids=str)
@pytest.mark.parametrize("grad_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_weight_gradients(shape, grad_dtype, accumulate):
    _backward(shape, "bf16", "silu", "same", grad_dtype=grad_dtype, accumulate=accumulate)


@pytest.mark.parametrize("dx,dw,again", [(True, False, False), (False, True, False), (False, False, True), (True, True, False)])
@pytest.mark.parametrize("saved", ["none", "same"])
def test_backward_of_some(dx, dw, again, saved):
    _backward((200, 136, 300, 0, 0), "bf16", "silu", saved, dx=dx, dw=dw, again=again)


def test_backward_of_many_tiles():
    """More tiles of each product than CTA pairs, of unlike costs; and products whose K goes round the ring many times."""
    for shape in ((2600, 2100, 600, 0, 0), (300, 2304, 2600, 0, 0), (9000, 520, 264, 0, 0)):
        _backward(shape, "bf16", "silu", "same", again=False)


def test_no_rows():
    w = torch.ones(5, 16, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(0, 5, dtype=torch.bfloat16, device="cuda")
    call = q.gated_ffn(none, w, w, h, 0, 16, 5, "bf16")
    ws = torch.empty(max(256, q.qmuon_gated_ffn_workspace_size(call)), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_forward(call, ws)
    for accumulate in (False, True):
        a, b = Matrix(5, 16, 3, torch.bfloat16), Matrix(5, 16, 3, torch.bfloat16)
        call = q.gated_ffn_grad(h, none, w, w, none, a.t, b.t, 0, 16, 5, "bf16", accumulate=accumulate, ld_dw_gate=a.ld, ld_dw_up=b.ld)
        q.qmuon_gated_ffn_backward(call, ws)
        torch.cuda.synchronize()
        for m in (a, b):
            m.check()
            assert bool((m.t == (3.0 if accumulate else 0.0)).all())


def test_values_that_are_not_finite_stay_in_their_rows():
    rows, width, inner = 300, 64, 256
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    w = [torch.randn(inner, width, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    clean = x.clone()
    x[7, 3], x[299, 0] = float("nan"), float("inf")
    hs = []
    for v in (clean, x):
        h = torch.empty(rows, inner, dtype=torch.bfloat16, device="cuda")
        call = q.gated_ffn(v, *w, h, rows, width, inner, "bf16")
        ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
        q.qmuon_gated_ffn_forward(call, ws)
        hs.append(h)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[7] = bad[299] = True
    assert torch.equal(hs[0][~bad], hs[1][~bad])
    assert bool(torch.isnan(hs[1][7]).all()) and not bool(torch.isfinite(hs[1][299]).any())


@pytest.mark.parametrize("name", ACTS)
def test_far_arguments(name):
    """gate far beyond where exp and the polynomials leave fp32's range: the activation is 0 or g, its slope 0 or 1."""
    g = torch.tensor([-3e38, -1e30, -1e10, -200.0, -30.0, 0.0, 30.0, 200.0, 1e10, 1e30, 3e38], device="cuda").bfloat16()
    n = g.numel()
    x, wg = torch.ones(1, 1, device="cuda").bfloat16(), g.view(n, 1).contiguous()
    wu = torch.ones(n, 1, device="cuda").bfloat16()
    h, dh = torch.empty(1, n, dtype=torch.bfloat16, device="cuda"), torch.ones(1, n, device="cuda").bfloat16()
    call = q.gated_ffn(x, wg, wu, h, 1, 1, n, "bf16", act=name)
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_forward(call, ws)
    want = torch.where(g > 0, g, torch.zeros_like(g))
    assert (h[0].double() - want.double()).abs().max() <= 1e-11         # silu(-30) = -2.8e-12
    dwg, dwu, again = torch.empty(n, 1, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 1, dtype=torch.bfloat16, device="cuda"), h.clone()
    call = q.gated_ffn_grad(dh, x, wg, wu, None, dwg, dwu, 1, 1, n, "bf16", act=name, h=again)
    ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_backward(call, ws)
    slope = torch.where(g > 0, 1.0, 0.0) + torch.where(g == 0, 0.5, 0.0)
    assert (dwg[:, 0].double() - slope.double()).abs().max() <= 1e-10 and torch.equal(dwu[:, 0], again[0]) and torch.equal(again, h)


def test_gradients_against_differences():
    """The block's own forward pass, moved the way the gradient points (a random direction can have next to no slope,
    and would show nothing); fp16 inputs on a grid that the steps stay on."""
    rows, width, inner = 40, 48, 64
    gen = torch.Generator("cuda").manual_seed(7)
    grid = lambda *s: torch.randint(-64, 65, s, generator=gen, device="cuda").float() / 64    # noqa: E731
    vals = [grid(rows, width), grid(inner, width) / 4, grid(inner, width) / 4]
    dh = grid(rows, inner)

    def value(v):
        x, wg, wu = (t.half() for t in v)
        assert all(torch.equal(a.float(), b) for a, b in zip((x, wg, wu), v))
        h = torch.empty(rows, inner, dtype=torch.float16, device="cuda")
        call = q.gated_ffn(x, wg, wu, h, rows, width, inner, "f16", act="gelu_tanh")
        ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
        q.qmuon_gated_ffn_forward(call, ws)
        return float((h.double() * dh.double()).sum()), float((h.double().abs() * dh.double().abs()).square().sum().sqrt())
    grads = [torch.empty(v.shape, dtype=torch.float16, device="cuda") for v in vals]
    call = q.gated_ffn_grad(dh.half(), *(v.half() for v in vals), *grads, rows, width, inner, "f16", act="gelu_tanh")
    ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_backward(call, ws)
    for k, g in enumerate(grads):
        step = g.float().sign() / (64 if k == 0 else 256)
        hi, n1 = value([v + step if i == k else v for i, v in enumerate(vals)])
        lo, n2 = value([v - step if i == k else v for i, v in enumerate(vals)])
        want = 2 * float((g.double() * step.double()).sum())
        # roundings of h: 6 standard deviations of independent ones of half a step at most; of the gradients likewise; and a
        # third of the third derivative of act(gate) up along the step (act's second is below 0.8, its third below 1.6)
        x, wg, wu = (v.double() for v in vals)
        s = step.double()
        zero = torch.zeros(rows, inner, dtype=torch.float64, device="cuda")
        dg, du = ((s @ wg.T, s @ wu.T), (x @ s.T, zero), (zero, x @ s.T))[k]
        third = float((dh.double().abs() * (1.6 * dg.abs() ** 3 * ((x @ wu.T).abs() + du.abs()) + 2.4 * dg ** 2 * du.abs())).sum()) / 3
        tol = 6 * 2.0 ** -11 * (n1 + n2) + 6 * 2.0 ** -10 * float((g.double() * s).square().sum().sqrt()) * 2 + third
        assert abs(hi - lo - want) <= tol, (k, hi - lo, want, tol)
        assert tol < 0.1 * abs(want)


def test_calls_repeat_bit_for_bit_and_in_graphs():
    shape = (300, 200, 392)
    gen = torch.Generator("cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()   # noqa: E731
    rows, width, inner = shape
    x, wg, wu, dh = rnd(rows, width), rnd(inner, width), rnd(inner, width), rnd(rows, inner)
    outs = [[torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, inner), (rows, width), (inner, width), (inner, width))]
            for _ in range(2)]
    pairs, sizes = [], []
    for h, dx, a, b in outs:
        f, g = q.gated_ffn(x, wg, wu, h, *shape, "bf16"), q.gated_ffn_grad(dh, x, wg, wu, dx, a, b, *shape, "bf16")
        pairs.append((f, g))
        sizes += [q.qmuon_gated_ffn_workspace_size(f), q.qmuon_gated_ffn_backward_workspace_size(g)]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def both(k):
        q.qmuon_gated_ffn_forward(pairs[k][0], ws)
        q.qmuon_gated_ffn_backward(pairs[k][1], ws)
    both(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):          # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(1)
        graphs.append(g)
    for g in graphs * 2:
        for t in outs[1]:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_calls_on_two_streams_with_workspaces_of_their_own():
    gen = torch.Generator("cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()   # noqa: E731
    rows, width, inner = 700, 512, 768
    sets = [(rnd(rows, width), rnd(inner, width), rnd(inner, width)) for _ in range(2)]
    hs = [[torch.empty(rows, inner, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    calls = [[q.gated_ffn(*s, h, rows, width, inner, "bf16") for h in two] for s, two in zip(sets, hs)]
    wss = [torch.empty(q.qmuon_gated_ffn_workspace_size(c[0]), dtype=torch.uint8, device="cuda") for c in calls]
    for c, w in zip(calls, wss):
        q.qmuon_gated_ffn_forward(c[0], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, w, s in zip(calls, wss, streams):
            q.qmuon_gated_ffn_forward(c[1], w, stream=s)
    torch.cuda.synchronize()
    for a, b in hs:
        assert torch.equal(a, b)


def test_a_recorded_failure_is_reported_and_cleared():
    rows, width, inner = 300, 1024, 512
    x, w = torch.ones(rows, width, device="cuda").bfloat16(), torch.ones(inner, width, device="cuda").bfloat16()
    h = torch.empty(rows, inner, dtype=torch.bfloat16, device="cuda")
    call = q.gated_ffn(x, w, w, h, rows, width, inner, "bf16")
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_forward(call, ws)
    want = h.clone()
    ws[:8].view(torch.int32).copy_(torch.tensor([q.QMUON_ERR_TIMEOUT, 0x2300], dtype=torch.int32))    # as a kernel records it
    with pytest.raises(q.QmuonError) as e:
        q.qmuon_sync_status(ws)
    assert e.value.status == q.QMUON_ERR_TIMEOUT
    q.qmuon_sync_status(ws)
    # a record that nobody read does not stop the next call
    ws[:4].view(torch.int32).fill_(q.QMUON_ERR_TIMEOUT)
    h.fill_(0.0)
    q.qmuon_gated_ffn_forward(call, ws)
    q.qmuon_sync_status(ws)
    assert torch.equal(h, want)


def test_arrays_of_another_device_are_refused(monkeypatch):
    """The calls run on the current device; with one GPU here, the current one is said to be another."""
    t = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    tokens, byte = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4096, dtype=torch.uint8, device="cuda")
    call = q.gated_ffn(t, t, t, torch.empty(4, 4, dtype=torch.bfloat16, device="cuda"), 4, 64, 4, "bf16")
    grad = q.gated_ffn_grad(torch.empty(4, 4, dtype=torch.bfloat16, device="cuda"), t, t, t, t.clone(), None, None, 4, 64, 4, "bf16")
    monkeypatch.setattr(q, "_device", lambda: 1)
    for f in (lambda: q.qmuon_embedding_forward(t, tokens, t.clone(), 4, 4, 64, "bf16"),
              lambda: q.qmuon_embedding_backward(t, tokens, t.clone(), 4, 4, 64, "bf16", byte, ws_bytes=1 << 20),
              lambda: q.qmuon_mxfp8_encode(t, byte, byte, 4, 64, "bf16"), lambda: q.qmuon_mxfp8_decode(byte, byte, t, 4, 64, "bf16"),
              lambda: q.qmuon_gated_ffn_forward(call, byte), lambda: q.qmuon_gated_ffn_backward(grad, byte)):
        with pytest.raises(q.QmuonError) as e:
            f()
        assert e.value.status == q.QMUON_ERR_INVALID_ARGUMENT and "current device" in str(e.value)
