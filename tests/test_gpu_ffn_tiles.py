"""The gated block's projections on the tensor cores, by the tiles that a call
takes: 128 or 64 columns of gate and of up, forward and computed again in the
backward pass, finished by the product's own epilogue or through partial sums,
in one piece of K or several.  Which of them a size goes to is the library's
choice, so each test looks at the kernels that ran.  Bounds as in the tests of
the small sizes, whose projections go through the cores' registers."""

import re
import warnings

import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_embedding import DT
from test_gpu_ffn import _backward, _check_forward

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
TYPES = ["bf16", "f16"]
FWD, BWD = 0, 1
FROM_PART = 0
_profiles = False


def _ran(f):
    """(the call's result, [(kernel, its numbers)] of the gated block's kernels that it launched)."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        r = f()
        torch.cuda.synchronize()
    found = [re.search(r"::(ffn_kernel|elem_kernel|few_kernel)<([^>]*)>", e.name) for e in p.events()]
    return r, [(m.group(1), [{"true": 1, "false": 0}.get(v.strip()) if v.strip() in ("true", "false") else int(re.sub(r"\(.*?\)", "", v))
                             for v in m.group(2).split(",")]) for m in found if m]


@pytest.fixture(scope="module", autouse=True)
def _profiler_has_run():
    """A process's first profile shows torch's launches only.  Where no profile shows any kernel, because another tool holds the
    GPU's counters, the values are tested and the kernels are not looked at."""
    global _profiles
    x, w, h = (torch.ones(n, 8, dtype=torch.bfloat16, device="cuda") for n in (4, 8, 4))
    call = q.gated_ffn(x, w, w, h, 4, 8, 8, "bf16")
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        _, kernels = _ran(lambda: q.qmuon_gated_ffn_forward(call, ws))
    _profiles = bool(kernels)
    if not _profiles:
        warnings.warn("torch.profiler shows no kernels here: which of them ran is not tested")


def _went(kernels, kind, dtype, name, columns, joined):
    """The projections went by tiles of `columns` columns; `joined`: and through partial sums, not straight to the results."""
    if not _profiles:
        return
    tiles = [k for n, k in kernels if n == "ffn_kernel" and k[0] == kind]
    assert tiles == [[kind, TYPES.index(dtype), ACTS.index(name), columns]], kernels
    assert any(n == "elem_kernel" and k[2] == FROM_PART for n, k in kernels) == joined, kernels
    assert not any(n == "few_kernel" for n, _ in kernels)


# shape (rows, width, inner, pad, off), columns of a tile, through partial sums.  Of either width: more tiles than pairs or
# ragged in every size; K round the ring of shared memory; K in pieces; rows that leave by elements
TILES = [((513, 136, 5984, 0, 0), 128, False), ((600, 1032, 3008, 0, 8), 128, False), ((1000, 4104, 224, 0, 0), 128, True),
         ((3001, 64, 2016, 3, 1), 128, True), ((257, 1100, 416, 0, 0), 64, False), ((1000, 520, 224, 8, 0), 64, False),
         ((260, 2056, 192, 0, 0), 64, True), ((129, 2001, 320, 3, 1), 64, True)]
BOTH = [("bf16", "silu"), ("f16", "gelu"), ("bf16", "gelu_tanh"), ("f16", "silu"), ("bf16", "gelu"), ("f16", "gelu_tanh")]


@pytest.mark.parametrize("shape,columns,joined", TILES, ids=str)
@pytest.mark.parametrize("i", range(6), ids=lambda k: "-".join(BOTH[k]))
def test_forward(shape, columns, joined, i):
    dtype, name = BOTH[i]
    saved = ("mxfp8", "same", "none", "none", "same", "mxfp8")[i]
    _, kernels = _ran(lambda: _check_forward(shape, dtype, name, saved))
    _went(kernels, FWD, dtype, name, columns, joined)


@pytest.mark.parametrize("shape,columns,joined", TILES, ids=str)
@pytest.mark.parametrize("i", range(6), ids=lambda k: "-".join(BOTH[k]))
def test_backward_from_nothing_kept(shape, columns, joined, i):
    dtype, name = BOTH[i]
    _, kernels = _ran(lambda: _backward(shape, dtype, name, "none", again=i % 2 == 0))
    _went(kernels, BWD, dtype, name, columns, joined)


@pytest.mark.parametrize("shape", [(513, 160, 5984, 0, 0), (257, 1120, 416, 0, 0)], ids=str)
def test_backward_from_a_carrier_of_x(shape):
    _, kernels = _ran(lambda: _backward(shape, "bf16", "silu", "none", x_mxfp8=True))
    _went(kernels, BWD, "bf16", "silu", 128 if shape[0] == 513 else 64, False)


# one of each width, unsplit and written by the epilogue
DIRECT = [((3001, 64, 2016), 128), ((1000, 520, 224), 64)]


def _operands(shape, dtype="bf16", seed=4):
    rows, width, inner = shape
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    x, wg, wu = rnd(rows, width), rnd(inner, width) * width ** -0.5, rnd(inner, width) * width ** -0.5
    return [t.to(DT[dtype]) for t in (x, wg, wu, rnd(rows, inner))]


def _run_forward(x, wg, wu, shape, dtype="bf16", name="silu", saved="none"):
    rows, width, inner = shape
    kept = {}
    if saved == "same":
        kept = {k: torch.empty(rows, inner, dtype=DT[dtype], device="cuda") for k in ("gate", "up")}
    elif saved == "mxfp8":
        kept = {k: torch.empty(rows, n, dtype=torch.uint8, device="cuda")
                for k, n in (("gate", inner), ("up", inner), ("gate_scale", inner // 32), ("up_scale", inner // 32))}
    h = torch.empty(rows, inner, dtype=DT[dtype], device="cuda")
    call = q.gated_ffn(x, wg, wu, h, rows, width, inner, dtype, act=name, saved=saved, **kept)
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_forward(call, ws)
    q.qmuon_sync_status(ws)
    return h, kept


def _run_backward(x, wg, wu, dh, shape, dtype="bf16", name="silu", dw=True):
    rows, width, inner = shape
    dx, h = torch.empty_like(x), torch.empty_like(dh)
    dwg, dwu = (torch.empty_like(wg), torch.empty_like(wu)) if dw else (None, None)
    call = q.gated_ffn_grad(dh, x, wg, wu, dx, dwg, dwu, rows, width, inner, dtype, act=name, h=h)
    ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=torch.uint8, device="cuda")
    q.qmuon_gated_ffn_backward(call, ws)
    q.qmuon_sync_status(ws)
    return dx, dwg, dwu, h


@pytest.mark.parametrize("shape,columns", DIRECT, ids=str)
@pytest.mark.parametrize("saved", ["same", "mxfp8"])
def test_values_that_are_not_finite_stay_in_their_rows(shape, columns, saved):
    """Rows on both sides of the tiles' and the CTAs' borders, and the last."""
    rows = shape[0]
    x, wg, wu, dh = _operands(shape)
    clean, kept = _run_forward(x, wg, wu, shape, saved=saved)
    clean_dx, _, _, clean_h = _run_backward(x, wg, wu, dh, shape, dw=False)
    x = x.clone()
    nan, inf = [127, 255, rows - 1], [128, 256]
    for r in nan:
        x[r, r % shape[1]] = float("nan")
    for r in inf:
        x[r, r % shape[1]] = float("inf")
    good = torch.ones(rows, dtype=torch.bool, device="cuda")
    good[nan + inf] = False
    (h, after), kernels = _ran(lambda: _run_forward(x, wg, wu, shape, saved=saved))
    _went(kernels, FWD, "bf16", "silu", columns, False)
    (dx, _, _, again), kernels = _ran(lambda: _run_backward(x, wg, wu, dh, shape, dw=False))
    _went(kernels, BWD, "bf16", "silu", columns, False)
    for a, b in ((h, clean), (dx, clean_dx), (again, clean_h), *((after[k], kept[k]) for k in kept)):
        assert torch.equal(a[good], b[good])
    assert bool(torch.isnan(h[nan]).all()) and not bool(torch.isfinite(h[~good]).any()) and not bool(torch.isfinite(again[~good]).any())
    assert not bool(torch.isfinite(dx[~good]).any())


@pytest.mark.parametrize("shape,columns", DIRECT, ids=str)
def test_weights_that_are_not_finite_stay_in_their_columns(shape, columns):
    inner = shape[2]
    x, wg, wu, _ = _operands(shape)
    clean, _ = _run_forward(x, wg, wu, shape)
    wg, wu = wg.clone(), wu.clone()
    bad = [31, 64, 127, 128, inner - 1]
    wg[bad[:3], 5] = float("nan")
    wu[bad[3:], 7] = float("nan")
    (h, _), kernels = _ran(lambda: _run_forward(x, wg, wu, shape))
    _went(kernels, FWD, "bf16", "silu", columns, False)
    good = torch.ones(inner, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert torch.equal(h[:, good], clean[:, good]) and bool(torch.isnan(h[:, ~good]).all())


@pytest.mark.parametrize("shape,columns", DIRECT, ids=str)
@pytest.mark.parametrize("name", ACTS)
def test_far_arguments(shape, columns, name):
    """gate far beyond where exp and the polynomials leave fp32's range: the activation is 0 or g, its slope 0 or 1.  dh is
    one row's, the last: the weights' gradients are the slopes and the activations themselves."""
    rows, width, inner = shape
    g = torch.tensor([-3e38, -1e30, -1e10, -200.0, -30.0, 0.0, 30.0, 200.0, 1e10, 1e30, 3e38], device="cuda").bfloat16()
    g = g.repeat(-(-inner // g.numel()))[:inner]
    x, wg, wu, dh = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((rows, width), (inner, width), (inner, width), (rows, inner)))
    x[:, 0], wg[:, 0], wu[:, 0], dh[-1] = 1.0, g, 1.0, 1.0
    (h, _), kernels = _ran(lambda: _run_forward(x, wg, wu, shape, name=name))
    _went(kernels, FWD, "bf16", name, columns, False)
    want = torch.where(g > 0, g, torch.zeros_like(g))
    assert (h[0].double() - want.double()).abs().max() <= 1e-11         # silu(-30) = -2.8e-12
    assert torch.equal(h, h[:1].expand_as(h))
    (_, dwg, dwu, again), kernels = _ran(lambda: _run_backward(x, wg, wu, dh, shape, name=name))
    _went(kernels, BWD, "bf16", name, columns, False)
    slope = torch.where(g > 0, 1.0, 0.0) + torch.where(g == 0, 0.5, 0.0)
    assert (dwg[:, 0].double() - slope.double()).abs().max() <= 1e-10
    assert torch.equal(dwu[:, 0], h[0]) and torch.equal(again, h)
    assert not bool(dwg[:, 1:].any()) and not bool(dwu[:, 1:].any())


@pytest.mark.parametrize("shape,columns", [((600, 1032, 3008), 128), ((1000, 520, 192), 64)], ids=str)
def test_gradients_against_differences(shape, columns):
    """The forward pass moved the way the gradient points, on a grid that fp16 inputs stay on."""
    rows, width, inner = shape
    gen = torch.Generator("cuda").manual_seed(7)
    grid = lambda *s: torch.randint(-64, 65, s, generator=gen, device="cuda").float() / 64    # noqa: E731
    vals = [grid(rows, width), grid(inner, width) / 16, grid(inner, width) / 16]
    dh = grid(rows, inner)

    def value(v):
        x, wg, wu = (t.half() for t in v)
        assert all(torch.equal(a.float(), b) for a, b in zip((x, wg, wu), v))
        h, _ = _run_forward(x, wg, wu, shape, "f16", "gelu_tanh")
        return float((h.double() * dh.double()).sum()), float((h.double().abs() * dh.double().abs()).square().sum().sqrt())
    (dx, dwg, dwu, _), kernels = _ran(lambda: _run_backward(*(v.half() for v in vals), dh.half(), shape, "f16", "gelu_tanh"))
    _went(kernels, BWD, "f16", "gelu_tanh", columns, False)
    for k, g in enumerate((dx, dwg, dwu)):
        step = g.float().sign() / (64 if k == 0 else 1024)
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
        assert tol < 0.01 * abs(want)


@pytest.mark.parametrize("shape,columns", [((513, 136, 5984), 128), ((257, 1100, 416), 64), ((1000, 4104, 224), 128)], ids=str)
def test_calls_repeat_bit_for_bit_and_in_graphs(shape, columns):
    rows, width, inner = shape
    x, wg, wu, dh = _operands(shape, seed=8)
    outs = [[torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, inner), (rows, width), (inner, width), (inner, width))]
            for _ in range(2)]
    pairs = [(q.gated_ffn(x, wg, wu, h, *shape, "bf16"), q.gated_ffn_grad(dh, x, wg, wu, dx, a, b, *shape, "bf16")) for h, dx, a, b in outs]
    ws = torch.empty(max(max(q.qmuon_gated_ffn_workspace_size(f), q.qmuon_gated_ffn_backward_workspace_size(g)) for f, g in pairs),
                     dtype=torch.uint8, device="cuda")

    def both(k):
        q.qmuon_gated_ffn_forward(pairs[k][0], ws)
        q.qmuon_gated_ffn_backward(pairs[k][1], ws)
    _, kernels = _ran(lambda: both(0))
    for kind in (FWD, BWD) if _profiles else ():
        assert [k[3] for n, k in kernels if n == "ffn_kernel" and k[0] == kind] == [columns]
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
    q.qmuon_sync_status(ws)
