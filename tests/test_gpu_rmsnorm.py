"""The RMS norm on the GPU against fp64: rows from one element to ones longer
than a CTA's registers, odd widths, strides and starts, guard bytes around what
is written.

u = 2^-24, ut the stored type's unit roundoff.  A row's sum of squares has at
most 40 additions on any path for rows that fit (96 for the longest ones here,
whose threads add up to 64 each), halved by the root; with the division, the
root and three products that is under 64 u of y.  h itself carries one rounding.
"""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import carrier, training

from gpu_util import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 1e-40, "f16": 2.0 ** -25, "f32": 1e-44}
# rows, cols, pad: one row and many, every way a row is split over threads, and rows read twice
SHAPES = [(1, 1, 0), (5, 7, 0), (3, 32, 0), (300, 64, 0), (1000, 128, 8), (33, 100, 3), (64, 1000, 0), (7, 2049, 0),
          (5, 4096, 0), (1, 4096, 0), (700, 4096, 0), (9, 5120, 16), (4, 16384, 0), (3, 8191, 0), (2, 8200, 1), (2, 40000, 0), (2, 33001, 7)]


class Matrix:
    """rows x cols of a guarded buffer, rows ld = cols + pad apart, `off` elements in."""

    def __init__(self, rows, cols, pad, dtype, off=0, fill=None):
        self.g = Guarded((rows * (cols + pad) + off,), dtype)
        self.g.t.fill_(3.0)
        self.ld = cols + pad
        self.t = self.g.t[off:].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.t.copy_(fill)
        self.pad = self.g.t[off:].view(rows, self.ld)[:, cols:]
        self.off = off

    def check(self):
        self.g.check()
        assert bool((self.pad == 3.0).all()) and bool((self.g.t[:self.off] == 3.0).all())


def _np(t):
    return t.detach().cpu().double().numpy()


def _rnd(gen, rows, cols, scale=1.0):
    col = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.02, 20.0, 1.0) * scale
    return torch.randn(rows, cols, generator=gen, device="cuda") * col


def _forward(rows, cols, pad, dtype, residual, off, alias=False, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DT[dtype]
    x = Matrix(rows, cols, pad, dt, off, _rnd(gen, rows, cols))
    r = Matrix(rows, cols, pad, dt, off, _rnd(gen, rows, cols, 2.0)) if residual else None
    gain = torch.randn(cols + 4, generator=gen, device="cuda")[off % 4:][:cols]
    s = x if alias else Matrix(rows, cols, pad, dt, off)
    y = Matrix(rows, cols, pad, dt, off)
    want = training.rmsnorm64(_np(x.t), _np(gain), 1e-5, _np(r.t) if residual else None)
    mag = np.abs(_np(x.t)) + (np.abs(_np(r.t)) if residual else 0)
    q.qmuon_rmsnorm_forward(x.t, gain, rows, cols, dtype, 1e-5, y=y.t, residual=r.t if residual else None, sum=s.t, ld_x=x.ld,
                            ld_residual=x.ld, ld_sum=s.ld, ld_y=y.ld)
    torch.cuda.synchronize()
    for m in (x, s, y) + ((r,) if residual else ()):
        m.check()
    return want, s, y, mag


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual,off,alias", [(True, 0, False), (False, 0, False), (True, 1, True)])
def test_forward(shape, dtype, residual, off, alias):
    (h, y), s, out, mag = _forward(*shape, dtype, residual, off, alias)
    ut = UT[dtype]
    assert (np.abs(_np(s.t) - h) <= ut * np.abs(h) * (1 + U) + U * mag + TINY[dtype]).all()
    assert (np.abs(_np(out.t) - y) <= (ut + 64 * U) * np.abs(y) + TINY[dtype]).all()


@pytest.mark.parametrize("shape", [(1, 32, 0), (3, 64, 0), (500, 128, 0), (7, 4096, 0), (65, 2048, 8), (9, 96, 3), (5, 2080, 1), (2, 40000, 0),
                                   (2, 33024, 7)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("both", [False, True])
def test_forward_mxfp8(shape, dtype, both):
    rows, cols, pad = shape
    gen = torch.Generator("cuda").manual_seed(2)
    x = Matrix(rows, cols, pad, DT[dtype], 0, _rnd(gen, rows, cols))
    x.t[rows // 2, :32] = 0.0           # a block of zeros
    gain = torch.randn(cols, generator=gen, device="cuda") * torch.exp2(torch.randint(-20, 20, (cols,), generator=gen, device="cuda").float())
    y = Matrix(rows, cols, pad, DT[dtype]) if both and dtype != "f16" else None
    pay, sc = Guarded((rows, cols), torch.uint8), Guarded((rows, cols // 32), torch.uint8)
    q.qmuon_rmsnorm_forward(x.t, gain, rows, cols, dtype, 1e-5, y=y.t if y else None, payload=pay.t, scale_inv=sc.t, ld_x=x.ld,
                            ld_y=y.ld if y else None)
    torch.cuda.synchronize()
    pay.check()
    sc.check()
    x.check()
    _, want = training.rmsnorm64(_np(x.t), _np(gain), 1e-5)
    if y:
        y.check()
        assert (np.abs(_np(y.t) - want) <= (UT[dtype] + 64 * U) * np.abs(want) + TINY[dtype]).all()
    byte = sc.t.cpu().numpy().astype(np.int64)
    top = np.abs(want.reshape(rows, -1, 32)).max(2)
    scale = 2.0 ** (byte - 127)
    assert (byte[top == 0] == 127).all()
    nz = top > 0
    # the smallest power of two that leaves the maximum within 448
    assert (top[nz] <= 448 * scale[nz] * (1 + 64 * U)).all() and (top[nz] > 224 * scale[nz] * (1 - 64 * U)).all()
    got = carrier.e4m3_decode(pay.t.cpu().numpy().reshape(-1)).reshape(rows, cols) * np.repeat(scale, 32, 1)
    # half a step: 2^-4 of the value, 2^-10 of the scale below the normal range; the fp32 error may move it by a little more
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 64 * U) + 2.0 ** -10 * np.repeat(scale, 32, 1)).all()
    assert (np.abs(got) <= 448 * np.repeat(scale, 32, 1)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [32, 64, 96, 160, 512, 1056, 4096, 9984, 16384])
@pytest.mark.parametrize("pay_off,offs", [(1, (0, 0, 0)), (2, (1, 2, 3)), (8, (3, 0, 1)), (0, (0, 1, 0))])
def test_forward_mxfp8_from_anywhere(dtype, cols, pay_off, offs):
    # payloads at any address, inputs that start unlike each other.  Bounds: test_forward_mxfp8's, with h's rounding in both terms
    rows, pads = 19 if cols < 4096 else 5, (1, 4, 3)
    gen = torch.Generator("cuda").manual_seed(13)
    x, r = _rnd(gen, rows, cols).to(DT[dtype]), _rnd(gen, rows, cols).to(DT[dtype])
    gain = torch.randn(cols, generator=gen, device="cuda")
    X, R, S = (Matrix(rows, cols, p, DT[dtype], o, f) for p, o, f in zip(pads, offs, (x, r, None)))
    pay, sc = Guarded((rows * cols + pay_off,), torch.uint8), Guarded((rows, cols // 32), torch.uint8)
    pay.t[:pay_off] = 7
    q.qmuon_rmsnorm_forward(X.t, gain, rows, cols, dtype, 1e-5, residual=R.t, sum=S.t, payload=pay.t[pay_off:], scale_inv=sc.t, ld_x=X.ld,
                            ld_residual=R.ld, ld_sum=S.ld)
    torch.cuda.synchronize()
    for m in (X, R, S, pay, sc):
        m.check()
    assert bool((pay.t[:pay_off] == 7).all())
    h, want = training.rmsnorm64(_np(x), _np(gain), 1e-5, _np(r))
    mag = (np.abs(_np(x)) + np.abs(_np(r))) / np.sqrt(np.mean(h * h, 1, keepdims=True)) * np.abs(_np(gain))
    assert (np.abs(_np(S.t) - h) <= UT[dtype] * np.abs(h) * (1 + U) + U * (np.abs(_np(x)) + np.abs(_np(r))) + TINY[dtype]).all()
    top = np.abs(want.reshape(rows, -1, 32)).max(2)
    err = 64 * U * top + (U * mag).reshape(rows, -1, 32).max(2)
    scale = 2.0 ** (sc.t.cpu().numpy().astype(np.int64) - 127)
    assert (top <= 448 * scale + err).all() and (top > 224 * scale - err).all()
    scale = np.repeat(scale, 32, 1)
    got = carrier.e4m3_decode(pay.t[pay_off:].cpu().numpy()).reshape(rows, cols) * scale
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 64 * U) + 2 * U * mag + 2.0 ** -10 * scale).all()
    assert (np.abs(got) <= 448 * scale).all()


def test_forward_mxfp8_equals_the_carrier_of_y():
    # in fp32, the payload and scales are the carrier of the y that the same call stores
    rows, cols = 130, 1056
    gen = torch.Generator("cuda").manual_seed(3)
    x, gain = _rnd(gen, rows, cols), torch.randn(cols, generator=gen, device="cuda")
    y = torch.empty(rows, cols, device="cuda")
    pay, sc = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_forward(x, gain, rows, cols, "f32", 1e-5, y=y, payload=pay, scale_inv=sc)
    p, s = carrier.encode_rows(y.cpu().numpy())
    np.testing.assert_array_equal(pay.cpu().numpy(), p)
    np.testing.assert_array_equal(sc.cpu().numpy(), s)


def test_forward_rows_of_zeros_and_non_finite_rows():
    x = torch.randn(4, 256, device="cuda")
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    gain = torch.ones(256, device="cuda")
    y = torch.empty_like(x)
    pay, sc = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(4, 8, dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_forward(x, gain, 4, 256, "f32", 0.0, y=y, payload=pay, scale_inv=sc)
    y2 = torch.empty_like(x)
    q.qmuon_rmsnorm_forward(x, gain, 4, 256, "f32", 1e-5, y=y2)
    assert torch.isnan(y[0]).all() and (y2[0] == 0).all()      # 0 / 0 without eps
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all() and (y[2, 6:] == 0).all()
    assert torch.isfinite(y[3]).all()                           # other rows are not touched by it
    assert ((pay[1] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("shape", SHAPES + [(5000, 96, 0), (2500, 2048, 0)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dsum,off,alias", [(True, 0, None), (False, 0, None), (True, 1, "dsum"), (False, 0, "dy")])
def test_backward(shape, dtype, dsum, off, alias):
    rows, cols, pad = shape
    gen = torch.Generator("cuda").manual_seed(4)
    dt = DT[dtype]
    h, dy = Matrix(rows, cols, pad, dt, off, _rnd(gen, rows, cols)), Matrix(rows, cols, pad, dt, off, _rnd(gen, rows, cols, 0.1))
    ds = Matrix(rows, cols, pad, dt, off, _rnd(gen, rows, cols, 0.1)) if dsum else None
    gain = torch.randn(cols + 4, generator=gen, device="cuda")[off % 4:][:cols]
    dx = {None: None, "dsum": ds, "dy": dy}[alias] or Matrix(rows, cols, pad, dt, off)
    dg = Guarded((cols,), torch.float32)
    need = q.qmuon_rmsnorm_workspace_size(rows, cols)
    ws = Guarded((need,), torch.uint8)
    ws.t.fill_(0xFF)
    want, wg = training.rmsnorm_grad64(_np(dy.t), _np(h.t), _np(gain), 1e-5, _np(ds.t) if dsum else None)
    H, D, G, S = _np(h.t), np.abs(_np(dy.t)), np.abs(_np(gain)), np.abs(_np(ds.t)) if dsum else 0.0
    q.qmuon_rmsnorm_backward(dy.t, h.t, gain, rows, cols, dtype, 1e-5, dx.t, dg.t, ws.t, dsum=ds.t if dsum else None, ld_dy=dy.ld, ld_h=h.ld,
                             ld_dsum=dy.ld, ld_dx=dx.ld)
    torch.cuda.synchronize()
    for m in (h, dy, dx) + ((ds,) if dsum else ()):
        m.check()
    dg.check()
    ws.check()
    # 64 u of each term's magnitude, as for y, and again for the second sum; the stored type's rounding
    inv = 1 / np.sqrt(np.mean(H * H, 1, keepdims=True) + 1e-5)
    n = np.abs(H) * inv
    mag = inv * (D * G + n * np.mean(D * G * n, 1, keepdims=True))
    assert (np.abs(_np(dx.t) - want) <= UT[dtype] * (1 + U) * np.abs(want) + 128 * U * mag + U * (S + np.abs(want)) + TINY[dtype]).all()
    # n's 64 u, and the additions over rows: those of a thread, of a CTA and of the partial sums, under 96 here
    assert (np.abs(_np(dg.t) - wg) <= 160 * U * np.sum(D * n, 0) + 1e-44).all()


def test_backward_by_differences():
    # fp32 gradients against central differences of the fp64 loss
    rows, cols = 37, 640
    gen = torch.Generator("cuda").manual_seed(5)
    h, dy, ds, gain = _rnd(gen, rows, cols), _rnd(gen, rows, cols), _rnd(gen, rows, cols), torch.randn(cols, generator=gen, device="cuda")
    dx, dg = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_backward(dy, h, gain, rows, cols, "f32", 1e-5, dx, dg, ws, dsum=ds)
    H, D, S, G = _np(h), _np(dy), _np(ds), _np(gain)
    loss = lambda a, b: float(np.sum(D * training.rmsnorm64(a, b, 1e-5)[1]) + np.sum(S * a))   # noqa: E731
    rng = np.random.default_rng(6)
    for _ in range(4):
        a, b, e = rng.standard_normal((rows, cols)), rng.standard_normal(cols), 1e-5
        num = (loss(H + e * a, G + e * b) - loss(H - e * a, G - e * b)) / (2 * e)
        got = float(np.sum(_np(dx) * a) + np.sum(_np(dg) * b))
        assert abs(num - got) <= 1e-4 * (np.linalg.norm(_np(dx)) + np.linalg.norm(_np(dg)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [1, 7, 64, 100, 101, 128, 257, 513, 4096])
@pytest.mark.parametrize("rows", [1, 3, 801])
def test_backward_without_eps(dtype, cols, rows):
    # rows that a CTA has room for but that do not exist: 1 / sqrt(0) of theirs must not reach the gain's gradient.
    # Bounds: test_backward's
    gen = torch.Generator("cuda").manual_seed(12)
    h, dy = _rnd(gen, rows, cols).to(DT[dtype]), _rnd(gen, rows, cols).to(DT[dtype])
    h[h == 0] = 1.0
    gain = torch.randn(cols, generator=gen, device="cuda")
    dx, dg = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_backward(dy, h, gain, rows, cols, dtype, 0.0, dx, dg, ws)
    H, D, G = _np(h), _np(dy), _np(gain)
    wx, wg = training.rmsnorm_grad64(D, H, G, 0.0)
    inv = 1 / np.sqrt(np.mean(H * H, 1, keepdims=True))
    n, a = np.abs(H) * inv, np.abs(D * G)
    mag = inv * (a + n * np.mean(a * n, 1, keepdims=True))
    assert (np.abs(_np(dx) - wx) <= UT[dtype] * (1 + U) * np.abs(wx) + 128 * U * mag + U * np.abs(wx) + TINY[dtype]).all()
    assert (np.abs(_np(dg) - wg) <= 160 * U * np.sum(np.abs(D) * n, 0) + 1e-44).all()


def test_no_rows():
    dg = torch.full((64,), 7.0, device="cuda")
    ws = torch.empty(q.qmuon_rmsnorm_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    gain = torch.ones(64, device="cuda")
    x = torch.ones(1, 64, device="cuda")
    q.qmuon_rmsnorm_forward(x, gain, 0, 64, "f32", 1e-5, y=x)
    q.qmuon_rmsnorm_backward(x, x, gain, 0, 64, "f32", 1e-5, x, dg, ws)
    torch.cuda.synchronize()
    assert (dg == 0).all() and (x == 1).all()
    none = torch.empty(0, 64, device="cuda")      # its address is null
    q.qmuon_rmsnorm_forward(none, gain, 0, 64, "f32", 1e-5, y=none)
    q.qmuon_rmsnorm_backward(none, none, gain, 0, 64, "f32", 1e-5, none, dg.fill_(7.0), ws)
    assert (dg == 0).all()
    with pytest.raises(q.QmuonError) as err:
        q.qmuon_rmsnorm_backward(x, x, gain, 1, 64, "f32", 1e-5, x, dg, ws, ws_bytes=16)
    assert err.value.status == q.QMUON_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("dtype,shape", [("bf16", (3000, 4096)), ("f32", (40000, 128)), ("f16", (500, 2049))])
def test_streams_graphs_and_repeats_give_the_same_bits(dtype, shape):
    rows, cols = shape
    gen = torch.Generator("cuda").manual_seed(8)
    h, dy = _rnd(gen, rows, cols).to(DT[dtype]), _rnd(gen, rows, cols).to(DT[dtype])
    gain = torch.randn(cols, generator=gen, device="cuda")
    need = q.qmuon_rmsnorm_workspace_size(rows, cols)
    outs = []

    def call(stream=None):
        y, dx, dg = torch.empty_like(h), torch.empty_like(h), torch.empty(cols, device="cuda")
        ws = torch.full((need,), len(outs) * 85, dtype=torch.uint8, device="cuda")
        outs.append((y, dx, dg, ws))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        q.qmuon_rmsnorm_forward(h, gain, rows, cols, dtype, 1e-5, y=y, stream=stream)
        q.qmuon_rmsnorm_backward(dy, h, gain, rows, cols, dtype, 1e-5, dx, dg, ws, stream=stream)

    call()
    call()
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(outs[0][:3], o[:3]):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    rows, cols = (1 << 20) + 5, 4104
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, cols, device="cuda").to(torch.bfloat16)
    gain = torch.ones(cols, device="cuda")
    y = torch.empty_like(x)
    q.qmuon_rmsnorm_forward(x, gain, rows, cols, "bf16", 1e-5, y=y)
    _, want = training.rmsnorm64(_np(x[-3:]), np.ones(cols), 1e-5)
    assert (np.abs(_np(y[-3:]) - want) <= (UT["bf16"] + 64 * U) * np.abs(want)).all()
    assert not bool(y[:-3].any())
    dg = torch.empty(cols, device="cuda")
    ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_backward(x, x, gain, rows, cols, "bf16", 1e-5, y, dg, ws)
    dx, wg = training.rmsnorm_grad64(_np(x[-3:]), _np(x[-3:]), np.ones(cols), 1e-5)
    np.testing.assert_allclose(_np(dg), wg, rtol=160 * U)
    assert not bool(y[:-3].any())
    assert bool(y[-3:].any())


WIDTHS = list(range(1, 70)) + [96, 100, 127, 128, 129, 255, 256, 257, 300, 511, 512, 513, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 2050, 2052, 4095,
                               4096, 4098, 4100]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [3, 200])
def test_every_width(dtype, rows):
    # forward and backward of each width: fp64 as above
    gen = torch.Generator("cuda").manual_seed(9)
    ut = UT[dtype]
    for cols in WIDTHS:
        h, dy, ds = (_rnd(gen, rows, cols).to(DT[dtype]) for _ in range(3))
        gain = torch.randn(cols, generator=gen, device="cuda")
        y, dx, dg = torch.empty_like(h), torch.empty_like(h), torch.empty(cols, device="cuda")
        ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
        q.qmuon_rmsnorm_forward(h, gain, rows, cols, dtype, 1e-5, y=y)
        q.qmuon_rmsnorm_backward(dy, h, gain, rows, cols, dtype, 1e-5, dx, dg, ws, dsum=ds)
        H, D, G, S = _np(h), _np(dy), _np(gain), _np(ds)
        _, want = training.rmsnorm64(H, G, 1e-5)
        assert (np.abs(_np(y) - want) <= (ut + 64 * U) * np.abs(want) + TINY[dtype]).all(), cols
        wx, wg = training.rmsnorm_grad64(D, H, G, 1e-5, S)
        n = np.abs(H) / np.sqrt(np.mean(H * H, 1, keepdims=True) + 1e-5)
        inv = 1 / np.sqrt(np.mean(H * H, 1, keepdims=True) + 1e-5)
        a = np.abs(D * G)
        mag = inv * (a + n * np.mean(a * n, 1, keepdims=True))
        assert (np.abs(_np(dx) - wx) <= ut * (1 + U) * np.abs(wx) + 128 * U * mag + U * (np.abs(S) + np.abs(wx)) + TINY[dtype]).all(), cols
        assert (np.abs(_np(dg) - wg) <= 160 * U * np.sum(np.abs(D) * n, 0) + 1e-44).all(), cols


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 64, 100, 2049, 4100, 9001, 20004, 70003])
@pytest.mark.parametrize("pads,offs", [((0, 1, 2, 3), (0, 0, 0, 0)), ((1, 3, 1, 5), (0, 0, 0, 0)), ((4, 4, 12, 8), (0, 4, 0, 8)),
                                       ((2, 2, 6, 2), (2, 0, 2, 4)), ((8, 16, 0, 8), (1, 1, 1, 1)), ((0, 0, 0, 0), (1, 0, 3, 2))])
def test_arrays_with_strides_and_starts_of_their_own(dtype, cols, pads, offs):
    # each array has its own stride and start, guards around and between its rows; the numbers are those of contiguous arrays
    rows = 21 if cols < 9000 else 4
    gen = torch.Generator("cuda").manual_seed(10)
    dt, ut = DT[dtype], UT[dtype]
    x, r, d = (_rnd(gen, rows, cols).to(dt) for _ in range(3))
    gain = torch.randn(cols, generator=gen, device="cuda")
    X, R, S, Y = (Matrix(rows, cols, p, dt, o, f) for p, o, f in zip(pads, offs, (x, r, None, None)))
    q.qmuon_rmsnorm_forward(X.t, gain, rows, cols, dtype, 1e-5, y=Y.t, residual=R.t, sum=S.t, ld_x=X.ld, ld_residual=R.ld, ld_sum=S.ld, ld_y=Y.ld)
    h, want = training.rmsnorm64(_np(x), _np(gain), 1e-5, _np(r))
    assert (np.abs(_np(Y.t) - want) <= (ut + 64 * U) * np.abs(want) + TINY[dtype]).all()
    assert (np.abs(_np(S.t) - h) <= ut * np.abs(h) * (1 + U) + U * (np.abs(_np(x)) + np.abs(_np(r))) + TINY[dtype]).all()
    for m in (X, R, S, Y):
        m.check()
    D, H, T, O = (Matrix(rows, cols, p, dt, o, f) for p, o, f in zip(pads, offs, (d, x, r, None)))
    dg, ws = torch.empty(cols, device="cuda"), torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_rmsnorm_backward(D.t, H.t, gain, rows, cols, dtype, 1e-5, O.t, dg, ws, dsum=T.t, ld_dy=D.ld, ld_h=H.ld, ld_dsum=T.ld, ld_dx=O.ld)
    wx, wg = training.rmsnorm_grad64(_np(d), _np(x), _np(gain), 1e-5, _np(r))
    inv = 1 / np.sqrt(np.mean(_np(x) ** 2, 1, keepdims=True) + 1e-5)
    n, a = np.abs(_np(x)) * inv, np.abs(_np(d) * _np(gain))
    # the longest rows add up to 256 terms in a thread: four times the bound of the others
    k = 4 if cols > 20000 else 1
    mag = inv * (a + n * np.mean(a * n, 1, keepdims=True))
    assert (np.abs(_np(O.t) - wx) <= ut * (1 + U) * np.abs(wx) + 128 * k * U * mag + U * (np.abs(_np(r)) + np.abs(wx)) + TINY[dtype]).all()
    assert (np.abs(_np(dg) - wg) <= 160 * k * U * np.sum(np.abs(_np(d)) * n, 0) + 1e-44).all()
    for m in (D, H, T, O):
        m.check()
