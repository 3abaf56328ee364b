"""Workloads of the training operators beside the Muon step: global gradient
clipping, AdamW over many tensors (fp32 and 8-bit states) and the RMS norm
with its residual (forward, with a same-type or an MXFP8 output, and backward).

``listed()`` names the cases, ``draw()`` makes one more of the same ranges,
``prepare()`` makes what a training program holds before the call and
``run()`` makes the call: with elementary torch operations in fp32 where
``own`` is false, through ``memory_reduced_muon_gb300`` where it is true.
``exact()`` evaluates the definitions in fp64.
"""

import numpy as np
import torch

own = False

DEVICE = "cuda"
BLOCK = 256                       # elements of an 8-bit state block
T, LR, BETA1, BETA2, EPS_ADAM = 7, 1e-3, 0.9, 0.99, 1e-8
SEED_SR = 0x1234567890ABCDEF      # key of the stochastic rounding
EPS_NORM = 1e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}


def listed():
    return [
        # the norm gains and biases of a small model: latency, no scaling asked for
        dict(name="clip_small", op="clip", tensors=24, numel=4096, ragged=False, grad="f32", apply=False, fill=1.0),
        # every matrix gradient of a training step (872M elements), clipped in place
        dict(name="clip_matrices", op="clip", tensors=32, numel=27262976, ragged=False, grad="bf16", apply=True, fill=4.0),
        # the norm gains of a 32-layer model: 65 vectors, fp32 gradients as a norm's backward leaves them
        dict(name="adamw_gains", op="adamw", tensors=65, numel=4096, ragged=False, packed=False, grad="f32", copy="none", scaled=True),
        # parameters of all sizes laid end to end in flat buffers, so that most start off a 16-byte boundary
        dict(name="adamw_packed", op="adamw", tensors=201, numel=300001, ragged=True, packed=True, grad="bf16", copy="bf16", scaled=True),
        # a token embedding of 102400 rows with its bf16 working copy
        dict(name="adamw_embedding", op="adamw", tensors=1, numel=419430400, ragged=False, packed=False, grad="bf16", copy="bf16", scaled=True),
        # the same embedding with 8-bit states
        dict(name="adamw8_embedding", op="adamw8", tensors=1, numel=419430400, ragged=False, stochastic=False, grad="bf16", copy="bf16", scaled=True),
        # parameters of all sizes with 8-bit states, rounded stochastically
        dict(name="adamw8_ragged_sr", op="adamw8", tensors=101, numel=700001, ragged=True, stochastic=True, grad="f16", copy="none", scaled=False),
        # one token being generated
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, mxfp8=False, pad=0),
        # a batch of prompts, its output in 8 bits for the next product
        dict(name="norm_prompts_mxfp8", op="norm", rows=16384, cols=4096, dtype="bf16", residual=True, mxfp8=True, pad=0),
        # odd width and row stride in fp16
        dict(name="norm_odd", op="norm", rows=6001, cols=2049, dtype="f16", residual=True, mxfp8=False, pad=14),
        # the backward pass of a training batch, with the gradient of the residual stream
        dict(name="norm_grad_batch", op="norm_grad", rows=16384, cols=4096, dtype="bf16", residual=True, pad=0),
        # many short rows in fp32: a norm over each head of 128
        dict(name="norm_grad_heads", op="norm_grad", rows=131072, cols=128, dtype="f32", residual=False, pad=0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm, ends included."""
    x = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, x))


def draw(rng):
    op = rng.choice(["clip", "adamw", "adamw8", "norm", "norm_grad"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 32, 16384)
        rows = min(_log(rng, 1, 65536), max(1, (1 << 26) // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.7,
                 pad=rng.choice([0, 0, rng.randrange(1, 65)]))
        if op == "norm":
            c["mxfp8"] = rng.random() < 0.5
            if c["mxfp8"]:
                c["cols"] = max(32, cols // 32 * 32)
        else:
            c["cols"] = cols if rng.random() < 0.5 else max(64, cols // 64 * 64)
        return c
    tensors = _log(rng, 1, 300)
    most = {"clip": 1 << 28, "adamw": 1 << 27, "adamw8": 1 << 26}[op]
    numel = _log(rng, 1, max(1, min(1 << 26, most // tensors)))
    c = dict(op=op, tensors=tensors, numel=numel, ragged=rng.random() < 0.6, grad=rng.choice(["bf16", "f16", "f32"]))
    if op == "clip":
        c.update(apply=rng.random() < 0.5, fill=round(rng.uniform(0.5, 4.0), 3))
        return c
    c.update(copy=rng.choice(["none", "bf16", "f16"]), scaled=rng.random() < 0.5)
    if op == "adamw":
        c["packed"] = rng.random() < 0.5
    else:
        c["stochastic"] = rng.random() < 0.5
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def sizes(case):
    """Elements of each tensor: all alike, or spread over [1, numel]."""
    n = case["numel"]
    if not case["ragged"]:
        return [n] * case["tensors"]
    return [1 + (n - 1) * (i * 619 % 1009) // 1008 for i in range(case["tensors"])]


def _starts(ns, packed):
    """Where each tensor starts in its flat buffer, and the buffer's length:
    end to end, or each on a multiple of 256 elements."""
    step = np.asarray(ns if packed else [-(-n // BLOCK) * BLOCK for n in ns], dtype=np.int64)
    ends = np.cumsum(step)
    return (ends - step).tolist(), int(ends[-1])


def _keep(ns, starts, total):
    """True where a flat position belongs to a tensor (else padding); None if all do."""
    if sum(ns) == total:
        return None
    edge = torch.zeros(total + 1, dtype=torch.int8, device=DEVICE)
    edge[torch.tensor(starts, device=DEVICE)] += 1
    edge[torch.tensor([s + n for s, n in zip(starts, ns)], device=DEVICE)] -= 1
    return torch.cumsum(edge[:-1], 0, dtype=torch.int8).bool()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _gradient(g, total, keep, dtype, scale=1e-3):
    """Gradients of lognormal scale per 256 elements; a third of these runs is
    zero, as the rows of an embedding whose tokens did not occur."""
    nb = -(-total // BLOCK)
    s = torch.exp(_normal(g, nb, 1)) * scale
    s[torch.rand(nb, 1, generator=g, device=DEVICE) < 1 / 3] = 0.0
    x = _normal(g, nb, BLOCK).mul_(s).view(-1)[:total]
    if keep is not None:
        x = torch.where(keep, x, 0.0)
    return x.to(DT[dtype])


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    st = {"case": case}
    if own:
        import memory_reduced_muon_gb300 as q
        st["q"] = q
    return {"clip": _prepare_clip, "adamw": _prepare_adamw, "adamw8": _prepare_adamw,
            "norm": _prepare_norm, "norm_grad": _prepare_norm_grad}[case["op"]](case, g, st)


def _prepare_clip(case, g, st):
    ns = sizes(case)
    starts, total = _starts(ns, False)
    st["grad"] = _gradient(g, total, _keep(ns, starts, total), case["grad"], 1e-2)
    # the norm is about 1e-2 e sqrt(2 total / 3); `fill` times that is the norm before clipping to it
    st["max_norm"] = float(1e-2 * np.e * (total * 2 / 3) ** 0.5 / case["fill"])
    if own:
        q = st["q"]
        st["plan"] = q.qmuon_clip_plan_create([(st["grad"][s:s + n], case["grad"]) for s, n in zip(starts, ns)])
        st["ws"] = torch.empty(q.qmuon_clip_workspace_size(st["plan"]), dtype=torch.uint8, device=DEVICE)
        st["norm"] = torch.empty(2, device=DEVICE)
    return st


def _prepare_adamw(case, g, st):
    eight = case["op"] == "adamw8"
    ns = sizes(case)
    starts, total = _starts(ns, case.get("packed", False))
    keep = _keep(ns, starts, total)
    masked = lambda x: x if keep is None else torch.where(keep, x, 0.0)   # noqa: E731
    wd = [0.1 if i % 2 == 0 else 0.0 for i in range(len(ns))]
    scale = [0.5 if i % 3 == 2 else 1.0 for i in range(len(ns))]
    st["param"] = masked(_normal(g, total) * 0.02)
    st["grad"] = _gradient(g, total, keep, case["grad"])
    st["copy"] = torch.zeros(total, dtype=DT[case["copy"]], device=DEVICE) if case["copy"] != "none" else None
    st["coef"] = torch.full((1,), 0.73, device=DEVICE) if case["scaled"] else None
    if eight:
        # codes and block maxima as a few steps leave them: the largest code of a block is 448
        nb = total // BLOCK
        m = masked(_normal(g, total)).view(nb, BLOCK)
        r = masked(_normal(g, total).abs_() * torch.exp(_normal(g, total))).view(nb, BLOCK)
        st["m"] = (m * (448.0 / m.abs().amax(1, keepdim=True).clamp_min(1e-30))).to(torch.float8_e4m3fn).view(-1)
        st["v"] = (r * (448.0 / r.amax(1, keepdim=True).clamp_min(1e-30))).to(torch.float8_e4m3fn).view(-1)
        st["m_absmax"] = torch.exp(_normal(g, nb)) * 2e-3
        st["v_absmax"] = torch.exp(_normal(g, nb)) * 3e-3
    else:
        st["m"] = masked(_normal(g, total) * 1e-3)
        st["v"] = masked((_normal(g, total) * 1e-3).square_())
    # per-tensor decay and learning-rate factors, spread over the flat positions
    if len(ns) == 1:
        st["wd"], st["lr"] = torch.full((1,), wd[0], device=DEVICE), torch.full((1,), LR * scale[0], device=DEVICE)
    else:
        step = torch.tensor([b - a for a, b in zip(starts, starts[1:] + [total])], device=DEVICE)
        st["wd"] = torch.repeat_interleave(torch.tensor(wd, device=DEVICE), step)
        st["lr"] = torch.repeat_interleave(torch.tensor([LR * x for x in scale], device=DEVICE), step)
    if eight and case["stochastic"]:
        blocks = torch.tensor([-(-n // BLOCK) for n in ns], device=DEVICE)
        first = torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
        st["block_in_tensor"] = torch.arange(total // BLOCK, device=DEVICE) - first
        st["tensor_of_block"] = torch.repeat_interleave(torch.arange(len(ns), device=DEVICE), blocks)
    if own:
        q = st["q"]
        ts = []
        for i, (s, n) in enumerate(zip(starts, ns)):
            b0, b1 = s // BLOCK, -(-(s + n) // BLOCK)
            ts.append(q.adamw_tensor(
                st["param"][s:s + n], st["grad"][s:s + n], st["m"][s:s + n], st["v"][s:s + n], n, case["grad"],
                m_absmax=st["m_absmax"][b0:b1] if eight else None, v_absmax=st["v_absmax"][b0:b1] if eight else None,
                copy=None if st["copy"] is None else st["copy"][s:s + n],
                copy_dtype=case["copy"] if st["copy"] is not None else "bf16", weight_decay=wd[i], lr_scale=scale[i]))
        st["plan"] = q.qmuon_adamw_plan_create(ts, "e4m3" if eight else "f32")
    return st


def _rows(g, case, scale=1.0):
    """rows x cols values with a few wide columns, in rows of cols + pad elements."""
    ld = case["cols"] + case["pad"]
    col = torch.where(torch.rand(ld, generator=g, device=DEVICE) < 0.01, 20.0, 1.0) * scale
    return (_normal(g, case["rows"], ld) * col).to(DT[case["dtype"]])[:, :case["cols"]]


def _prepare_norm(case, g, st):
    rows, cols = case["rows"], case["cols"]
    st["x"] = _rows(g, case)
    st["residual"] = _rows(g, case, 3.0) if case["residual"] else None
    st["gain"] = 1.0 + 0.1 * _normal(g, cols)
    dt = DT[case["dtype"]]
    st["sum"] = torch.empty(rows, cols, dtype=dt, device=DEVICE) if case["residual"] else None
    if case["mxfp8"]:
        st["payload"] = torch.empty(rows, cols, dtype=torch.uint8, device=DEVICE)
        st["scale_inv"] = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEVICE)
    else:
        st["y"] = torch.empty(rows, cols, dtype=dt, device=DEVICE)
    return st


def _prepare_norm_grad(case, g, st):
    rows, cols = case["rows"], case["cols"]
    st["h"] = _rows(g, case, 2.0)
    st["dy"] = _rows(g, case, 1e-3)
    st["dsum"] = _rows(g, case, 1e-3) if case["residual"] else None
    st["gain"] = 1.0 + 0.1 * _normal(g, cols)
    if own:
        q = st["q"]
        st["dx"] = torch.empty(rows, cols, dtype=DT[case["dtype"]], device=DEVICE)
        st["dgain"] = torch.empty(cols, device=DEVICE)
        st["ws"] = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device=DEVICE)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_clip(s):
    q, c = s["q"], s["case"]
    q.qmuon_grad_clip(s["plan"], s["max_norm"], c["apply"], s["norm"], s["ws"])
    return {"norm": s["norm"][0], "coef": s["norm"][1], **({"grad": s["grad"]} if c["apply"] else {})}


def _own_adamw(s):
    q = s["q"]
    if s["case"].get("stochastic"):
        q.qmuon_adamw_step_sr(s["plan"], T, LR, BETA1, BETA2, EPS_ADAM, SEED_SR, s["coef"])
    else:
        q.qmuon_adamw_step(s["plan"], T, LR, BETA1, BETA2, EPS_ADAM, s["coef"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "copy", "m", "v", "m_absmax", "v_absmax") if s.get(k) is not None}


def _own_norm(s):
    q, c = s["q"], s["case"]
    r = s["residual"]
    q.qmuon_rmsnorm_forward(s["x"], s["gain"], c["rows"], c["cols"], c["dtype"], EPS_NORM, y=s.get("y"), residual=r,
                            sum=s["sum"], payload=s.get("payload"), scale_inv=s.get("scale_inv"),
                            ld_x=s["x"].stride(0), ld_residual=None if r is None else r.stride(0))
    out = {} if r is None else {"sum": s["sum"]}
    if c["mxfp8"]:
        # what the bytes stand for: E4M3 values and power-of-two scales
        return {**out, "payload": s["payload"].view(torch.float8_e4m3fn), "scale": s["scale_inv"].view(torch.float8_e8m0fnu)}
    return {**out, "y": s["y"]}


def _own_norm_grad(s):
    q, c = s["q"], s["case"]
    d = s["dsum"]
    q.qmuon_rmsnorm_backward(s["dy"], s["h"], s["gain"], c["rows"], c["cols"], c["dtype"], EPS_NORM, s["dx"], s["dgain"],
                             s["ws"], dsum=d, ld_dy=s["dy"].stride(0), ld_h=s["h"].stride(0),
                             ld_dsum=None if d is None else d.stride(0))
    return {"dx": s["dx"], "dgain": s["dgain"]}


def _plain_clip(s):
    g = s["grad"].float()
    norm = g.square().sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    if not s["case"]["apply"]:
        return {"norm": norm, "coef": coef}
    s["grad"].copy_(g * coef)
    return {"norm": norm, "coef": coef, "grad": s["grad"]}


def _scaled_gradient(s):
    g = s["grad"].float()
    return g if s["coef"] is None else g * s["coef"]


def _plain_update(s, m, root):
    """param and its copy from the new momentum and the square root of the new second moment."""
    c1, c2 = 1.0 - BETA1 ** T, 1.0 - BETA2 ** T
    step = s["lr"] * (1.0 / c1)
    p = s["param"] * (1.0 - s["lr"] * s["wd"]) - step * (m / (root * (1.0 / c2 ** 0.5) + EPS_ADAM))
    s["param"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)


def _plain_adamw(s):
    g = _scaled_gradient(s)
    m = s["m"] * BETA1 + g * (1.0 - BETA1)
    v = s["v"] * BETA2 + (g * g) * (1.0 - BETA2)
    _plain_update(s, m, v.sqrt())
    s["m"].copy_(m)
    s["v"].copy_(v)
    return _adamw_outputs(s)


def _words(s):
    """One Philox4x32-10 word per element: key = the seed, counter = (element / 4 in the tensor, its high part, the
    tensor's index, the step)."""
    lo = 0xFFFFFFFF
    j = (s["block_in_tensor"][:, None] * (BLOCK // 4) + torch.arange(BLOCK // 4, device=DEVICE)).view(-1)
    c = [j & lo, j >> 32, s["tensor_of_block"].repeat_interleave(BLOCK // 4), torch.full_like(j, T)]
    k = [SEED_SR & lo, SEED_SR >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # modulo 2^64: the low and high words of the products are right
        c = [((b >> 32) & lo) ^ c[1] ^ k[0], b & lo, ((a >> 32) & lo) ^ c[3] ^ k[1], a & lo]
        k = [(k[0] + 0x9E3779B9) & lo, (k[1] + 0xBB67AE85) & lo]
    return torch.stack(c, 1).view(-1, BLOCK)


def _to_e4m3(x, random16):
    """E4M3 of x (|x| <= 448): nearest, or up with the probability of the remainder where 16 random bits per value are
    given.  2^-120 x has the exponent field of E4M3, so its bits above the lowest 20 are the code, subnormals too."""
    if random16 is None:
        return x.to(torch.float8_e4m3fn)
    bits = (x.abs() * 2.0 ** -120).view(torch.int32)
    code = ((bits + (random16 << 4)) >> 20).clamp(max=0x7E)
    return (code | torch.where(x < 0, 0x80, 0)).to(torch.uint8).view(torch.float8_e4m3fn)


def _plain_adamw8(s):
    g = _scaled_gradient(s)
    blocks = lambda x: x.view(-1, BLOCK)   # noqa: E731
    f448 = torch.full((), 448.0, device=DEVICE)
    m_old = blocks(s["m"]).float() * (s["m_absmax"] / f448)[:, None]
    r_old = blocks(s["v"]).float() * (s["v_absmax"] / f448)[:, None]
    g = blocks(g)
    m = m_old * BETA1 + g * (1.0 - BETA1)
    root = ((r_old * r_old) * BETA2 + (g * g) * (1.0 - BETA2)).sqrt()
    _plain_update(s, m.view(-1), root.view(-1))
    m_max, r_max = m.abs().amax(1), root.amax(1)
    big = torch.finfo(torch.float32).max
    m_scaled = m * (f448 / m_max).clamp(max=big)[:, None]
    r_scaled = root * (f448 / r_max).clamp(max=big)[:, None]
    w = _words(s).to(torch.int64) if s["case"]["stochastic"] else None
    s["m"].copy_(_to_e4m3(m_scaled, None if w is None else (w & 0xFFFF).int()).view(-1))
    s["v"].copy_(_to_e4m3(r_scaled, None if w is None else (w >> 16).int()).view(-1))
    s["m_absmax"].copy_(m_max)
    s["v_absmax"].copy_(r_max)
    return _adamw_outputs(s)


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS_NORM) * s["gain"]
    out = {}
    if s["residual"] is not None:
        out["sum"] = h.to(DT[c["dtype"]])
    if not c["mxfp8"]:
        return {**out, "y": y.to(DT[c["dtype"]])}
    y = y.view(c["rows"], c["cols"] // 32, 32)
    amax = y.abs().amax(2, keepdim=True)
    f, e = torch.frexp(amax)                        # amax = f 2^e, f in [0.5, 1); 448 = 0.875 2^9
    byte = torch.where(amax == 0, 127, (e - 9 + 127 + (f > 0.875)).clamp(0, 254))
    payload = torch.ldexp(y, 127 - byte).to(torch.float8_e4m3fn).view(c["rows"], c["cols"])
    return {**out, "payload": payload, "scale": byte.to(torch.uint8).view(c["rows"], -1).view(torch.float8_e8m0fnu)}


def _plain_norm_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    inv = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS_NORM)
    n, a = h * inv, dy * s["gain"]
    dx = inv * (a - n * (a * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(DT[s["case"]["dtype"]]), "dgain": (dy * n).sum(0)}


_OWN = {"clip": _own_clip, "adamw": _own_adamw, "adamw8": _own_adamw, "norm": _own_norm, "norm_grad": _own_norm_grad}
_PLAIN = {"clip": _plain_clip, "adamw": _plain_adamw, "adamw8": _plain_adamw8, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size = case["rows"] * case["cols"], SIZE[case["dtype"]]
        if op == "norm":
            move = n * size * (3 if case["residual"] else 1) + (n + n // 32 if case["mxfp8"] else n * size)
            return {"bytes": move + 4 * case["cols"], "flops": 5 * n}
        return {"bytes": n * size * (4 if case["residual"] else 3) + 8 * case["cols"], "flops": 11 * n}
    n = sum(sizes(case))
    g = SIZE[case["grad"]]
    if op == "clip":
        return {"bytes": n * g * (2 if case["apply"] else 1) + 8, "flops": n * (3 if case["apply"] else 2)}
    nb = sum(-(-k // BLOCK) for k in sizes(case))
    state = 16 * n if op == "adamw" else 4 * n + 16 * nb
    return {"bytes": n * (8 + g + SIZE[case["copy"]]) + state, "flops": n * (16 if op == "adamw" else 22)}


# --------------------------------------------------------------------------
# the definitions in fp64
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"clip": _exact_clip, "adamw": _exact_adamw, "adamw8": _exact_adamw, "norm": _exact_norm,
            "norm_grad": _exact_norm_grad}[case["op"]](case, s)


def _exact_clip(case, s):
    g = s["grad"].double()
    norm = torch.linalg.vector_norm(g)
    coef = torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + 1e-6))
    return {"norm": norm, "coef": coef, **({"grad": g.mul_(coef)} if case["apply"] else {})}


def _exact_adamw(case, s):
    g = s["grad"].double()
    if case["scaled"]:
        g *= s["coef"].double()
    if case["op"] == "adamw8":
        unit = lambda a: a.double().div_(448).repeat_interleave(BLOCK)   # noqa: E731
        m0 = s["m"].double().mul_(unit(s["m_absmax"]))
        v0 = s["v"].double().mul_(unit(s["v_absmax"])).square_()
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m = m0.lerp_(g, 1.0 - BETA1)
    v = v0.lerp_(g.square_(), 1.0 - BETA2)
    lr = s["lr"].double()
    p = s["param"].double()
    p = p - lr * (s["wd"].double() * p + (m / (1.0 - BETA1 ** T)) / ((v / (1.0 - BETA2 ** T)).sqrt() + EPS_ADAM))
    out = {"param": p}
    if s["copy"] is not None:
        out["copy"] = p
    if case["op"] == "adamw":
        return {**out, "m": m, "v": v}
    words = _exact_words(case) if case["stochastic"] else None
    for key, x, shift in (("m", m, 0), ("v", v.sqrt_(), 16)):
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1)
        x = x * torch.where(top > 0, 448 / top, 0.0)[:, None]
        u = None if words is None else torch.from_numpy(((words >> shift) & 0xFFFF).astype(np.float64) / 65536).to(x.device).view_as(x)
        out[key], out[key + "_absmax"] = _exact_e4m3(x, u).view(-1), top
    return out


def _exact_e4m3(x, u=None):
    """x to the grid of E4M3 (3 mantissa bits, exponents from -6 up, largest 448): to the nearest, ties to even, or, with
    u in [0, 1), up where the remainder and u make a whole step."""
    grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    k = x / grid
    k = torch.round(k) if u is None else torch.sign(k) * torch.floor(k.abs() + u)
    return (k * grid).clamp_(-448, 448)


def _exact_words(case):
    """Philox4x32-10 words of the case's flat positions, tensor by tensor, with unsigned 64-bit products."""
    out = []
    for i, n in enumerate(sizes(case)):
        j = np.arange(-(-n // BLOCK) * BLOCK // 4, dtype=np.uint64)
        a, b, c, d = j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, i), np.full_like(j, T)
        for r in range(10):
            k0 = np.uint64((SEED_SR + r * 0x9E3779B9) & 0xFFFFFFFF)
            k1 = np.uint64(((SEED_SR >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
            x, y = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
            a, b, c, d = (y >> np.uint64(32)) ^ b ^ k0, y & np.uint64(0xFFFFFFFF), (x >> np.uint64(32)) ^ d ^ k1, x & np.uint64(0xFFFFFFFF)
        out.append(np.stack([a, b, c, d], 1).reshape(-1))
    return np.concatenate(out).astype(np.int64)


def _exact_norm(case, s):
    h = s["x"].double()
    if case["residual"]:
        h = h + s["residual"].double()
    y = s["gain"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + EPS_NORM)
    out = {"sum": h} if case["residual"] else {}
    if not case["mxfp8"]:
        return {**out, "y": y}
    y = y.view(case["rows"], -1, 32)
    top = y.abs().amax(2, keepdim=True)
    # the smallest power of two that leaves the largest of 32 values within 448
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), 0.0).clamp(-127, 127)
    return {**out, "payload": _exact_e4m3(y * torch.exp2(-e)).view(case["rows"], -1), "scale": torch.exp2(e).view(case["rows"], -1)}


def _exact_norm_grad(case, s):
    h, dy, gain = s["h"].double(), s["dy"].double(), s["gain"].double()
    w = h.square().sum(1, keepdim=True) / case["cols"] + EPS_NORM
    a = dy * gain
    dx = a * w.pow(-0.5) - h * (a * h).sum(1, keepdim=True) * w.pow(-1.5) / case["cols"]
    if case["residual"]:
        dx = dx + s["dsum"].double()
    return {"dx": dx, "dgain": (dy * h * w.pow(-0.5)).sum(0)}
