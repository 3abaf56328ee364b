"""AdamW over many tensors and gradient clipping on the GPU, against fp64
(fp32 states, norms) and bit for bit against the fp32 definition (8-bit
states).  Sizes from one element up, starts off every alignment, guard bytes
around everything that is written.

u = 2^-24 below.  Tolerances follow from one rounding per operation:
* g' = s g: u;  m: each product at most 3 u (constant, g', product) and the sum
  u, so 4 u of A = b1 |m| + (1 - b1) |g'|, 5 u with the higher orders;
* v >= 0, no cancellation: 2 u (g') doubled by the square... 6 u, 7 u taken;
* p: u per operation of p (1 - lr wd): 3 u |p| and the last sum, 4 u (|p| + |U|);
  U = step m / d: step 3 u, d: v's 7 u halved by the root, the root, its factor,
  the factor's own rounding, eps and the sum: 8 u, the division and the product:
  14 u |U|, and m's absolute error 5 u A step / d.
"""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import carrier, training

from gpu_util import Guarded, to_oracle_grad

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = [1, 3, 255, 256, 257, 2047, 2048, 2049, 5000, 70001]


def _np(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def _offset(n, dtype, off):
    """A tensor of n elements that starts `off` elements into a guarded buffer."""
    g = Guarded((n + off,), dtype)
    g.t.zero_()
    return g, g.t[off:]


def _f32_case(sizes, grad, copy, off, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=gen, device="cuda")   # noqa: E731
    ts, guards, descs = [], [], []
    for i, n in enumerate(sizes):
        d = {}
        for key, dt, val in (("param", torch.float32, rnd(n)), ("grad", DT[grad], rnd(n) * 1e-2), ("m", torch.float32, rnd(n) * 1e-2),
                             ("v", torch.float32, (rnd(n) * 1e-2).square())):
            g, d[key] = _offset(n, dt, off)
            d[key].copy_(val)
            guards.append(g)
        g, d["copy"] = _offset(n, DT[copy or "bf16"], off)
        guards.append(g)
        d["wd"], d["ls"] = (0.1, 0.0, 0.03)[i % 3], (1.0, 0.5)[i % 2]
        descs.append(q.adamw_tensor(d["param"], d["grad"], d["m"], d["v"], n, grad, copy=d["copy"] if copy else None,
                                    copy_dtype=copy or "bf16", weight_decay=d["wd"], lr_scale=d["ls"]))
        ts.append(d)
    return ts, guards, q.qmuon_adamw_plan_create(descs, "f32")


@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("grad,copy", [("bf16", "bf16"), ("f16", None), ("f32", "f16")])
def test_adamw_f32(grad, copy, off):
    t, lr, b1, b2, eps, s = 3, 1e-2, 0.9, 0.99, 1e-8, 0.37
    ts, guards, plan = _f32_case(SIZES, grad, copy, off, 7 + off)
    before = [{k: _np(d[k]) for k in ("param", "grad", "m", "v")} for d in ts]
    q.qmuon_adamw_step(plan, t, lr, b1, b2, eps, torch.full((1,), s, device="cuda"))
    torch.cuda.synchronize()
    s = float(np.float32(s))
    for d, b in zip(ts, before):
        p, m, v = training.adamw64(b["param"], b["grad"], b["m"], b["v"], t, lr * d["ls"], b1, b2, eps, d["wd"], s)
        A = b1 * np.abs(b["m"]) + (1 - b1) * np.abs(b["grad"] * s)
        assert (np.abs(_np(d["m"]) - m) <= 5 * U * A + 1e-44).all()
        assert (np.abs(_np(d["v"]) - v) <= 7 * U * v + 1e-44).all()
        den = (np.sqrt(v / (1 - b2 ** t)) + eps)
        step = lr * d["ls"] / (1 - b1 ** t)
        up = np.abs(step * m / den)
        assert (np.abs(_np(d["param"]) - p) <= 4 * U * (np.abs(p) + np.abs(b["param"])) + 20 * U * up + 6 * U * A * step / den).all()
        assert torch.equal(d["grad"].float().double().cpu(), torch.from_numpy(b["grad"]))   # read only
        want = d["param"].to(DT[copy]) if copy else torch.zeros_like(d["copy"])
        assert torch.equal(d["copy"], want)
    for g in guards:
        g.check()


def _e4m3_case(sizes, grad, copy, off, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=gen, device="cuda")   # noqa: E731
    ts, guards, descs = [], [], []
    for i, n in enumerate(sizes):
        nb = -(-n // 256)
        gr = rnd(n) * 1e-2 * torch.exp(rnd(n))
        gr[256:512] = 0.0
        code = lambda: torch.randint(0, 0x7F, (n,), generator=gen, device="cuda").to(torch.uint8)   # noqa: E731
        sign = (torch.randint(0, 2, (n,), generator=gen, device="cuda") * 128).to(torch.uint8)
        d = {}
        for key, dt, val, o in (("param", torch.float32, rnd(n), off), ("grad", DT[grad], gr, off), ("m", torch.uint8, code() | sign, 0),
                                ("v", torch.uint8, code(), 0), ("m_absmax", torch.float32, torch.exp(rnd(nb)) * 1e-2, off),
                                ("v_absmax", torch.float32, torch.exp(rnd(nb)) * 1e-2, off),
                                ("copy", DT[copy or "bf16"], torch.zeros(n, device="cuda"), off)):
            g, d[key] = _offset(val.numel(), dt, o)
            d[key].copy_(val)
            guards.append(g)
        d["wd"], d["ls"], d["n"] = (0.1, 0.0)[i % 2], (1.0, 0.5)[i % 2], n
        descs.append(q.adamw_tensor(d["param"], d["grad"], d["m"], d["v"], n, grad, d["m_absmax"], d["v_absmax"],
                                    d["copy"] if copy else None, copy or "bf16", d["wd"], d["ls"]))
        ts.append(d)
    return ts, guards, q.qmuon_adamw_plan_create(descs, "e4m3")


def _same_codes(a, b):
    nan = (b & 0x7F) == 0x7F
    np.testing.assert_array_equal((a & 0x7F)[nan], b[nan] & 0x7F)
    va, vb = carrier.e4m3_decode(a), carrier.e4m3_decode(b)
    np.testing.assert_array_equal(va[~nan], vb[~nan])   # -0 equals 0


def _check_e4m3(ts, host, t, lr, b1, b2, eps, s, seed):
    for i, (d, h) in enumerate(zip(ts, host)):
        p, m, v, mm, vm = training.adamw_e4m3(h["param"], h["grad"], h["m"], h["v"], h["m_absmax"], h["v_absmax"], t, lr, b1, b2,
                                              eps, d["wd"], d["ls"], s, seed, i)
        _same_codes(d["m"].cpu().numpy(), m)
        _same_codes(d["v"].cpu().numpy(), v)
        np.testing.assert_array_equal(d["m_absmax"].cpu().numpy(), mm)
        np.testing.assert_array_equal(d["v_absmax"].cpu().numpy(), vm)
        # the update may use an approximate quotient: p within 4 u |p| and 8 u of the update
        got = d["param"].cpu().numpy()
        ok = ~np.isnan(p)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(p))
        up = np.abs(p.astype(np.float64) - h["param"])
        assert (np.abs(got[ok].astype(np.float64) - p[ok]) <= (4 * U * (np.abs(p) + np.abs(h["param"])) + 8 * U * up)[ok]).all()


def _host(ts):
    return [{k: (d[k].float() if k == "grad" else d[k]).cpu().numpy().copy() for k in
             ("param", "grad", "m", "v", "m_absmax", "v_absmax")} for d in ts]


@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("grad,copy", [("bf16", "bf16"), ("f16", None), ("f32", "f16")])
def test_adamw_e4m3(grad, copy, sr, off):
    t, lr, b1, b2, eps, s, seed = 5, 1e-2, 0.9, 0.99, 1e-8, float(np.float32(0.37)), 0xFEDCBA9876543210
    ts, guards, plan = _e4m3_case(SIZES, grad, copy, off, 11 + off)
    scale = torch.full((1,), s, device="cuda")
    for k in range(2):   # the second step starts from the first one's states
        host = _host(ts)
        if sr:
            q.qmuon_adamw_step_sr(plan, t + k, lr, b1, b2, eps, seed, scale)
        else:
            q.qmuon_adamw_step(plan, t + k, lr, b1, b2, eps, scale)
        torch.cuda.synchronize()
        _check_e4m3(ts, host, t + k, lr, b1, b2, eps, s, seed if sr else None)
    for d in ts:
        if copy:
            assert torch.equal(d["copy"], d["param"].to(DT[copy]))
    for g in guards:
        g.check()


@pytest.mark.parametrize("sr", [False, True])
def test_adamw_e4m3_first_step_and_non_finite(sr):
    # a first step from zero bytes, with a NaN, an infinity, tiny and all-zero blocks among the gradients
    n = 256 * 5
    ts, guards, plan = _e4m3_case([n], "f32", None, 0, 3)
    d = ts[0]
    for k in ("m", "v", "m_absmax", "v_absmax"):
        d[k].zero_()
    g = torch.randn(n, device="cuda") * 1e-2
    g[5] = float("nan")
    g[256 + 7] = float("inf")
    g[512:768] *= 1e-38      # maxima below 448 / FLT_MAX
    g[768:1024] = 0.0
    d["grad"].copy_(g)
    for t in (1, 2):
        host = _host(ts)
        if sr:
            q.qmuon_adamw_step_sr(plan, t, 1e-2, 0.9, 0.99, 1e-8, 9)
        else:
            q.qmuon_adamw_step(plan, t, 1e-2, 0.9, 0.99, 1e-8)
        torch.cuda.synchronize()
        _check_e4m3(ts, host, t, 1e-2, 0.9, 0.99, 1e-8, 1.0, 9 if sr else None)
    assert torch.isfinite(d["param"][512:]).all()
    assert torch.isnan(d["param"][:256]).sum() == 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_a_scale_that_is_not_finite_changes_nothing(state, bad):
    ts, guards, plan = (_f32_case if state == "f32" else _e4m3_case)([300, 5000], "bf16", "bf16", 0, 5)
    before = [g.raw.clone() for g in guards]
    q.qmuon_adamw_step(plan, 1, 1e-2, 0.9, 0.99, 1e-8, torch.full((1,), bad, device="cuda"))
    torch.cuda.synchronize()
    for g, b in zip(guards, before):
        assert torch.equal(g.raw, b)


def test_stochastic_step_of_an_f32_plan_and_bad_steps_are_refused():
    ts, _, plan = _f32_case([100], "bf16", None, 0, 1)
    before = ts[0]["param"].clone()
    with pytest.raises(q.QmuonError) as e:
        q.qmuon_adamw_step_sr(plan, 1, 1e-2, 0.9, 0.99, 1e-8, 1)
    assert e.value.status == q.QMUON_ERR_UNSUPPORTED
    for a in ((0, 1e-2, 0.9, 0.99, 1e-8), (1, float("nan"), 0.9, 0.99, 1e-8), (1, 1e-2, 1.0, 0.99, 1e-8),
              (1, 1e-2, 0.9, -0.1, 1e-8), (1, 1e-2, 0.9, 0.99, 0.0), (1, 1e-2, 0.9, 0.99, 1e-60)):
        with pytest.raises(q.QmuonError) as e:
            q.qmuon_adamw_step(plan, *a)
        assert e.value.status == q.QMUON_ERR_INVALID_ARGUMENT, a
    torch.cuda.synchronize()
    assert torch.equal(before, ts[0]["param"])


def test_streams_graphs_and_repeats_give_the_same_bits():
    cases = [_e4m3_case(SIZES, "bf16", "bf16", 0, 21) for _ in range(3)]
    run = lambda plan, t, stream=None: q.qmuon_adamw_step_sr(plan, t, 1e-2, 0.9, 0.99, 1e-8, 4, stream=stream)   # noqa: E731
    for t in (1, 2):
        run(cases[0][2], t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (1, 2):
        run(cases[1][2], t, side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t in (1, 2):
            run(cases[2][2], t)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(*(x[1] for x in cases)):
        assert torch.equal(a.raw, b.raw) and torch.equal(a.raw, c.raw)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_offsets_past_32_bits(state):
    # only the first and last elements carry gradients; everything between stays zero
    n = (1 << 32) + 777
    z = lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")   # noqa: E731
    nb = -(-n // 256)
    st = z(n, torch.uint8 if state == "e4m3" else torch.float32), z(n, torch.uint8 if state == "e4m3" else torch.float32)
    mx = (z(nb, torch.float32), z(nb, torch.float32)) if state == "e4m3" else (None, None)
    p, g = z(n, torch.float32), z(n, torch.bfloat16)
    g[:1000] = 1.0
    g[-1000:] = -1.0
    plan = q.qmuon_adamw_plan_create([q.adamw_tensor(p, g, *st, n, "bf16", *mx)], state)
    clip = q.qmuon_clip_plan_create([(g, "bf16")])
    norm = torch.empty(2, device="cuda")
    ws = torch.empty(q.qmuon_clip_workspace_size(clip), dtype=torch.uint8, device="cuda")
    q.qmuon_grad_clip(clip, 1e9, False, norm, ws)
    q.qmuon_adamw_step(plan, 1, 0.5, 0.9, 0.99, 1e-8)
    # a first step moves each by lr g / (|g| + eps)
    np.testing.assert_allclose(p[:1000].cpu().numpy(), -0.5, rtol=1e-6)
    np.testing.assert_allclose(p[-1000:].cpu().numpy(), 0.5, rtol=1e-6)
    assert int((p != 0).sum()) == 2000
    assert abs(norm[0].item() - 2000 ** 0.5) <= 1e-6 * 2000 ** 0.5 and norm[1].item() == 1.0


# ---------------------------------------------------------------------------
# clipping
# ---------------------------------------------------------------------------
# a square and at most 12 additions of positive terms in fp32 (fp64 from there
# on), halved by the root, and the norm's own rounding: 8 u; the coefficient
# adds three roundings

def _clip_case(sizes, off, seed, scale=1e-2):
    gen = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        name = ("bf16", "f16", "f32")[i % 3]
        g, t = _offset(n, DT[name], off)
        t.copy_(torch.randn(n, generator=gen, device="cuda") * scale)
        out.append((g, t, name))
    return out


def _clip(case, max_norm, apply):
    plan = q.qmuon_clip_plan_create([(t, name) for _, t, name in case])
    ws = torch.full((q.qmuon_clip_workspace_size(plan),), 0xFF, dtype=torch.uint8, device="cuda")
    norm = Guarded((2,), torch.float32)
    q.qmuon_grad_clip(plan, max_norm, apply, norm.t, ws)
    torch.cuda.synchronize()
    norm.check()
    return norm.t.cpu().numpy().astype(np.float64), plan, ws


@pytest.mark.parametrize("off", [0, 1, 4, 8])
@pytest.mark.parametrize("sizes", [[1], [0, 5], [8191, 8192, 8193], SIZES, [4096] * 300, [3_000_001]])
@pytest.mark.parametrize("fill", [0.5, 4.0])
def test_clip(sizes, off, fill):
    case = _clip_case(sizes, off, 3)
    before = [t.clone() for _, t, _ in case]
    want, _ = training.clip64([_np(t) for t in before], 1.0)
    max_norm = float(np.float32(want / fill))
    (norm, coef), _, _ = _clip(case, max_norm, False)
    _, c = training.clip64([_np(t) for t in before], max_norm)
    assert abs(norm - want) <= 8 * U * want
    assert abs(coef - c) <= 11 * U * c
    for b, (g, t, _) in zip(before, case):
        assert torch.equal(b, t)
    (norm2, coef2), _, _ = _clip(case, max_norm, True)
    assert (norm2, coef2) == (norm, coef)      # the same bits
    k = torch.tensor(coef, dtype=torch.float32, device="cuda")
    for b, (g, t, name) in zip(before, case):
        assert torch.equal(t, (b.float() * k).to(DT[name]) if coef < 1 else b)
        g.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_clip_of_a_gradient_that_is_not_finite(bad):
    case = _clip_case([5000, 300, 7], 0, 4)
    case[1][1][17] = bad
    before = [g.raw.clone() for g, _, _ in case]
    (norm, coef), _, _ = _clip(case, 1.0, True)
    assert not np.isfinite(norm) and np.isnan(coef)
    for b, (g, _, _) in zip(before, case):
        assert torch.equal(b, g.raw)           # left alone


def test_clip_of_zeros_and_refusals():
    case = _clip_case([5000], 0, 4, scale=0.0)
    (norm, coef), plan, ws = _clip(case, 1.0, True)
    assert norm == 0.0 and coef == 1.0
    n = torch.empty(4, device="cuda")
    for a, kw in (((0.0, False, n, ws), {}), ((-1.0, False, n, ws), {}), ((float("nan"), False, n, ws), {}), ((1.0, 2, n, ws), {}),
                  ((1.0, False, None, ws), {}), ((1.0, False, n, None), dict(ws_bytes=1 << 20))):
        with pytest.raises(q.QmuonError) as e:
            q.qmuon_grad_clip(plan, *a, **kw)
        assert e.value.status == q.QMUON_ERR_INVALID_ARGUMENT
    with pytest.raises(q.QmuonError) as e:
        q.qmuon_grad_clip(plan, 1.0, False, n, ws, ws_bytes=0)
    assert e.value.status == q.QMUON_ERR_WORKSPACE_TOO_SMALL


def test_clip_coefficient_feeds_the_step():
    # the coefficient read on the device gives what the scaled gradient gives
    ts, _, plan = _f32_case([5000, 77], "f32", None, 0, 31)
    us, _, plan2 = _f32_case([5000, 77], "f32", None, 0, 31)
    case = [(None, d["grad"], "f32") for d in ts]
    cplan = q.qmuon_clip_plan_create([(t, n) for _, t, n in case])
    ws = torch.empty(q.qmuon_clip_workspace_size(cplan), dtype=torch.uint8, device="cuda")
    norm = torch.empty(2, device="cuda")
    q.qmuon_grad_clip(cplan, 0.1, False, norm, ws)
    q.qmuon_adamw_step(plan, 1, 1e-2, 0.9, 0.99, 1e-8, norm[1:])
    for d in us:
        d["grad"].mul_(norm[1])
    q.qmuon_adamw_step(plan2, 1, 1e-2, 0.9, 0.99, 1e-8)
    for a, b in zip(ts, us):
        for k in ("param", "m", "v"):
            assert torch.equal(a[k], b[k])


@pytest.mark.parametrize("offs", [(1, 0, 2, 3, 0), (0, 1, 0, 0, 0), (2, 2, 2, 2, 1), (3, 3, 3, 3, 3), (1, 1, 1, 1, 5)])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_adamw_f32_arrays_at_offsets_of_their_own(grad, offs):
    # param, grad, m, v and copy start at different places: no head makes all of them aligned together (or one does)
    gen = torch.Generator("cuda").manual_seed(3)
    descs, ref, guards, ts = [], [], [], []
    for n in SIZES:
        vals = [torch.randn(n, generator=gen, device="cuda") * s for s in (1.0, 1e-2, 1e-2, 1e-2, 0.0)]
        vals[3] = vals[3].square()
        made = [_offset(n, dt, o) for dt, o in zip((torch.float32, DT[grad], torch.float32, torch.float32, torch.bfloat16), offs)]
        for (g, t), v in zip(made, vals):
            t.copy_(v)
            guards.append(g)
        p, g, m, v, c = (t for _, t in made)
        ts.append((p, m, v, c))
        descs.append(q.adamw_tensor(p, g, m, v, n, grad, copy=c, weight_decay=0.1))
        ref.append([t.clone() for t in (p, g, m, v)])
    q.qmuon_adamw_step(q.qmuon_adamw_plan_create(descs), 2, 1e-2, 0.9, 0.99, 1e-8)
    # the same numbers as aligned arrays give, bit for bit
    plain = [[t.clone() for t in r] for r in ref]
    q.qmuon_adamw_step(q.qmuon_adamw_plan_create([q.adamw_tensor(p, g, m, v, p.numel(), grad, weight_decay=0.1) for p, g, m, v in plain]),
                       2, 1e-2, 0.9, 0.99, 1e-8)
    for (p, m, v, c), (p1, _, m1, v1) in zip(ts, plain):
        assert torch.equal(p, p1) and torch.equal(m, m1) and torch.equal(v, v1) and torch.equal(c, p1.bfloat16())
    for g in guards:
        g.check()


def test_adamw_many_tensors_of_mixed_types():
    # 400 tensors, some of them empty, gradients of all types in one plan: each as if alone
    gen = torch.Generator("cuda").manual_seed(4)
    rnd = lambda n: torch.randn(n, generator=gen, device="cuda")   # noqa: E731
    made = []
    for i in range(400):
        n = (i * 37) % 3000
        name = ("bf16", "f16", "f32")[i % 3]
        made.append((rnd(n), (rnd(n) * 1e-2).to(DT[name]), rnd(n) * 1e-2, (rnd(n) * 1e-2).square(), name))
    alone = [[t.clone() for t in x[:4]] for x in made]
    desc = lambda t, name: q.adamw_tensor(*t, t[0].numel(), name, weight_decay=0.01)   # noqa: E731
    q.qmuon_adamw_step(q.qmuon_adamw_plan_create([desc(x[:4], x[4]) for x in made]), 3, 1e-2, 0.9, 0.99, 1e-8)
    for x, a in list(zip(made, alone))[::13]:
        if a[0].numel():
            q.qmuon_adamw_step(q.qmuon_adamw_plan_create([desc(a, x[4])]), 3, 1e-2, 0.9, 0.99, 1e-8)
            for s, t in zip(x[:4], a):
                assert torch.equal(s, t)


@pytest.mark.parametrize("sr", [False, True])
def test_adamw_e4m3_one_large_tensor_equals_many_launches_of_it(sr):
    # enough blocks for several per warp, against the same blocks as tensors of their own (nearest), or the oracle's
    # bits on a sample of them (stochastic: the counter holds the element's place)
    n, blk = 3 * 256 * 8 * 400, 256
    ts, guards, plan = _e4m3_case([n], "bf16", "bf16", 0, 9)
    host = _host(ts)
    if sr:
        q.qmuon_adamw_step_sr(plan, 4, 1e-2, 0.9, 0.99, 1e-8, 77)
    else:
        q.qmuon_adamw_step(plan, 4, 1e-2, 0.9, 0.99, 1e-8)
    torch.cuda.synchronize()
    d, h = ts[0], host[0]
    if sr:
        _check_e4m3(ts, host, 4, 1e-2, 0.9, 0.99, 1e-8, 1.0, 77)
    else:
        for b in range(0, n // blk, 997):
            s = slice(b * blk, (b + 1) * blk)
            p, m, v, mm, vm = training.adamw_e4m3(h["param"][s], h["grad"][s], h["m"][s], h["v"][s], h["m_absmax"][b:b + 1],
                                                  h["v_absmax"][b:b + 1], 4, 1e-2, 0.9, 0.99, 1e-8, d["wd"], d["ls"])
            _same_codes(d["m"][s].cpu().numpy(), m)
            _same_codes(d["v"][s].cpu().numpy(), v)
            assert d["m_absmax"][b].item() == mm[0] and d["v_absmax"][b].item() == vm[0]
    for g in guards:
        g.check()
