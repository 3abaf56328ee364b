"""Token embedding on the GPU: lookup and gradient against fp64, from one token
to many, tokens that are none, one token everywhere, rows of any start and
stride, guard bytes around what is written.

ut is the stored type's unit roundoff, u = 2^-24.  A looked-up value is one
product rounded once.  A row's gradient of n terms has n - 1 additions at most
one after another, one product and one rounding: |error| <= n u sum|terms| + ut
|value|."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import activations as act

from gpu_util import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 1e-40, "f16": 2.0 ** -25, "f32": 1e-44}


class Matrix:
    """rows x cols of a guarded buffer, rows cols + pad apart, `off` elements in; 3.0 around it."""

    def __init__(self, rows, cols, pad, dtype, off=0, fill=None):
        self.g = Guarded((max(rows, 1) * (cols + pad) + off,), dtype)
        self.g.t.fill_(3.0)
        self.ld, self.off = cols + pad, off
        self.rows = self.g.t[off:].view(max(rows, 1), self.ld)
        self.t = self.rows[:rows, :cols]
        if fill is not None:
            self.t.copy_(fill)

    def check(self):
        self.g.check()
        assert bool((self.rows[:, self.t.shape[1]:] == 3.0).all()) and bool((self.g.t[:self.off] == 3.0).all())


def _np(t):
    return t.detach().cpu().double().numpy()


def _tokens(n, vocab, kind, bits, gen):
    if kind == "one":
        t = torch.full((n,), vocab // 2, device="cuda")
    elif kind == "few":
        t = torch.randint(0, min(3, vocab), (n,), generator=gen, device="cuda")
    else:
        t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
        if kind == "holes":
            bad = torch.tensor([-1, vocab, 2 ** 31 - 1, -2 ** 31], device="cuda")
            t = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.3, bad[torch.randint(0, 4, (n,), generator=gen, device="cuda")], t)
            if n > 6:
                t[:3], t[-3:] = -1, vocab       # both ends
        if kind == "none":
            t.fill_(vocab)
    return t.to(torch.int64 if bits == 64 else torch.int32)


@pytest.mark.parametrize("n,vocab,cols,pad,off", [(1, 1, 1, 0, 0), (1, 7, 4096, 0, 0), (5, 9, 8, 0, 0), (33, 100, 257, 3, 1), (300, 50, 64, 8, 0),
                                                  (1000, 777, 100, 0, 2), (77, 20, 5000, 0, 0), (3, 4, 16384, 0, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits,scale", [(64, 1.0), (32, 22.6274)])
def test_lookup(n, vocab, cols, pad, off, dtype, bits, scale):
    gen = torch.Generator("cuda").manual_seed(n)
    table = Matrix(vocab, cols, pad, DT[dtype], off, torch.randn(vocab, cols, generator=gen, device="cuda"))
    tokens = _tokens(n, vocab, "holes", bits, gen)
    out = Matrix(n, cols, pad, DT[dtype], off)
    q.qmuon_embedding_forward(table.t, tokens, out.t, n, vocab, cols, dtype, scale=scale, ld_table=table.ld, ld_out=out.ld)
    torch.cuda.synchronize()
    out.check()
    table.check()
    want = act.embedding64(_np(table.t), tokens.cpu().numpy(), float(np.float32(scale)))
    assert (np.abs(_np(out.t) - want) <= UT[dtype] * np.abs(want) * (1 + U) + U * np.abs(want) + TINY[dtype]).all()
    if scale == 1.0:
        assert (_np(out.t) == want).all()


def test_lookup_takes_values_that_are_not_finite_only_from_its_rows():
    table = torch.full((4, 64), float("nan"), device="cuda")
    table[2] = 1.0
    table[3, 0] = float("inf")
    out = torch.full((4, 64), 7.0, device="cuda")
    q.qmuon_embedding_forward(table, torch.tensor([2, -1, 4, 3], device="cuda"), out, 4, 4, 64, "f32", scale=2.0)
    assert bool((out[0] == 2).all()) and bool((out[1:3] == 0).all()) and bool(torch.isinf(out[3, 0])) and bool(torch.isnan(out[3, 1]))


def _backward(n, vocab, cols, pad, off, dtype, grad_dtype, kind, bits, accumulate, seed=1, scale=0.75):
    gen = torch.Generator("cuda").manual_seed(seed)
    dout = Matrix(n, cols, pad, DT[dtype], off, torch.randn(n, cols, generator=gen, device="cuda"))
    tokens = _tokens(n, vocab, kind, bits, gen)
    before = torch.randn(vocab, cols, generator=gen, device="cuda")
    grad = Matrix(vocab, cols, pad, DT[grad_dtype], off, before)
    before = _np(grad.t)
    ws = Guarded((q.qmuon_embedding_workspace_size(n, vocab, cols),), torch.uint8)
    ws.t.fill_(0xFF)
    q.qmuon_embedding_backward(dout.t, tokens, grad.t, n, vocab, cols, dtype, ws.t, scale=scale, grad_dtype=grad_dtype,
                               accumulate=accumulate, ld_dout=dout.ld, ld_dtable=grad.ld)
    torch.cuda.synchronize()
    for m in (dout, grad, ws):
        m.check()
    want, mag, count = act.embedding_grad64(_np(dout.t), tokens.cpu().numpy(), vocab, scale)
    got = _np(grad.t)
    if accumulate:
        assert (got[count == 0] == before[count == 0]).all()
        want, mag = want + before, mag + np.abs(before)
    else:
        assert (got[count == 0] == 0).all()
    bound = (count[:, None] + 2) * U * mag + UT[grad_dtype] * np.abs(want) + TINY[grad_dtype]
    assert (np.abs(got - want) <= bound).all()
    return grad.t


# tokens, vocabulary, columns: one and many, pieces that end inside and at runs, vocabularies of one, two and three sorting passes
SHAPES = [(1, 1, 1, 0, 0), (1, 600, 64, 0, 0), (31, 5, 8, 0, 0), (32, 5, 64, 0, 0), (33, 511, 257, 3, 1), (64, 512, 128, 8, 0),
          (1000, 513, 100, 0, 0), (4096, 300, 64, 0, 0), (4097, 300, 72, 0, 8), (9001, 70000, 40, 0, 0), (12345, 300000, 16, 0, 0),
          (200, 90, 5000, 0, 0), (130, 40, 2064, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("kind,bits,accumulate", [("all", 64, False), ("holes", 32, True), ("holes", 64, False)])
def test_gradient(shape, dtype, grad_dtype, kind, bits, accumulate):
    _backward(*shape, dtype, grad_dtype, kind, bits, accumulate)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 96, 97, 1000, 4100, 20000])
@pytest.mark.parametrize("kind", ["one", "few", "none"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_long_runs(n, kind, accumulate):
    _backward(n, 10, 72, 0, 0, "bf16", "f32", kind, 64, accumulate)


@pytest.mark.parametrize("n,vocab,kind", [(8192, 600, "all"), (8193, 600, "holes"), (50001, 300000, "holes"), (65536, 500, "all"),
                                          (65537, 500, "all"), (131073, 90000, "holes"), (140000, 7, "one")])
def test_gradient_of_many_tokens(n, vocab, kind):
    """One CTA that sorts, clusters of them, and sorting by several kernels."""
    _backward(n, vocab, 8, 0, 0, "f32", "f32", kind, 64, False)


def test_gradient_of_very_wide_rows():
    """More columns than a grid's second dimension has slabs of 32, by elements and by vectors."""
    for cols, dtype in ((4200000 - 5701, "f32"), (4194304, "bf16")):
        n, vocab = 70, 2
        tokens = torch.cat([torch.zeros(66, dtype=torch.int64), torch.ones(4, dtype=torch.int64)]).cuda()
        dout = torch.ones(n, cols, dtype=DT[dtype], device="cuda")
        grad = torch.full((vocab, cols), 7.0, dtype=DT[dtype], device="cuda")
        ws = torch.empty(q.qmuon_embedding_workspace_size(n, vocab, cols), dtype=torch.uint8, device="cuda")
        q.qmuon_embedding_backward(dout, tokens, grad, n, vocab, cols, dtype, ws)
        assert bool((grad[0] == 66).all()) and bool((grad[1] == 4).all())
        out = torch.empty(n, cols, dtype=DT[dtype], device="cuda")
        q.qmuon_embedding_forward(grad, tokens, out, n, vocab, cols, dtype, scale=0.5)
        assert bool((out[:66] == 33).all()) and bool((out[66:] == 2).all())


def test_gradient_of_no_tokens():
    for accumulate in (False, True):
        _backward(0, 70, 72, 8, 0, "bf16", "bf16", "all", 64, accumulate)


def test_gradient_repeats_bit_for_bit():
    a = _backward(20000, 900, 200, 0, 0, "f32", "f32", "all", 64, False).clone()
    assert torch.equal(a, _backward(20000, 900, 200, 0, 0, "f32", "f32", "all", 64, False))


def test_gradient_takes_values_that_are_not_finite_only_to_their_rows():
    dout = torch.ones(100, 64, device="cuda")
    dout[7] = float("nan")
    tokens = torch.arange(100, device="cuda") % 9
    tokens[7] = 9
    tokens[8] = -1
    dout[8] = float("inf")
    grad = torch.empty(10, 64, device="cuda")
    ws = torch.empty(q.qmuon_embedding_workspace_size(100, 10, 64), dtype=torch.uint8, device="cuda")
    q.qmuon_embedding_backward(dout, tokens, grad, 100, 10, 64, "f32", ws)
    assert bool(torch.isnan(grad[9]).all()) and bool(torch.isfinite(grad[:9]).all())
    count = torch.bincount(tokens[tokens >= 0], minlength=10)[:9]
    assert torch.equal(grad[:9], count.float()[:, None].expand(9, 64))


def test_gradient_against_differences():
    gen = torch.Generator("cuda").manual_seed(5)
    table = torch.randn(20, 32, generator=gen, device="cuda")
    tokens = torch.randint(0, 20, (50,), generator=gen, device="cuda")
    weight = torch.randn(50, 32, generator=gen, device="cuda")       # of a linear function of the output
    grad = torch.empty_like(table)
    ws = torch.empty(q.qmuon_embedding_workspace_size(50, 20, 32), dtype=torch.uint8, device="cuda")
    q.qmuon_embedding_backward(weight, tokens, grad, 50, 20, 32, "f32", ws, scale=3.0)
    step = torch.randn(20, 32, generator=gen, device="cuda")

    def value(t):
        out = torch.empty(50, 32, device="cuda")
        q.qmuon_embedding_forward(t, tokens, out, 50, 20, 32, "f32", scale=3.0)
        return float((out.double() * weight.double()).sum())
    diff, want = value(table + step) - value(table), float((grad.double() * step.double()).sum())
    # the function is linear: 1600 products of fp32 roundings, a few units each, of magnitude 3 |t| |w|
    mag = float((3 * (table.abs() + step.abs()).double()[tokens] * weight.abs().double()).sum())
    assert abs(diff - want) <= 16 * U * mag


def test_captured_calls_and_another_stream():
    gen = torch.Generator("cuda").manual_seed(6)
    n, vocab, cols = 700, 90, 128
    dout = torch.randn(n, cols, generator=gen, device="cuda").bfloat16()
    tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    ws = torch.empty(q.qmuon_embedding_workspace_size(n, vocab, cols), dtype=torch.uint8, device="cuda")
    eager, grad, out = (torch.empty(s, cols, dtype=torch.bfloat16, device="cuda") for s in (vocab, vocab, n))
    q.qmuon_embedding_backward(dout, tokens, eager, n, vocab, cols, "bf16", ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q.qmuon_embedding_backward(dout, tokens, grad, n, vocab, cols, "bf16", ws)
        q.qmuon_embedding_forward(grad, tokens, out, n, vocab, cols, "bf16")
    for _ in range(3):
        grad.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, eager) and torch.equal(out, eager[tokens])
