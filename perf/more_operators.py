"""Workloads of the token embedding (lookup and gradient), the gated
feed-forward block (forward and backward) and the 8-bit activation checkpoints
(MXFP8 carriers of activations, and the backward pass that reads them).

``listed()`` names the cases, ``draw()`` makes one more of the same ranges,
``prepare()`` makes what a training program holds before the call and
``run()`` makes the call: with elementary torch operations in fp32 where
``own`` is false, through ``memory_reduced_muon_gb300`` where it is true.
``exact()`` evaluates the definitions in fp64.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one token being generated
        dict(name="embed_token", op="embed", tokens=1, vocab=102400, cols=4096, dtype="bf16", pad=0, scale=1.0),
        # a batch of prompts, rows scaled by the root of their width
        dict(name="embed_prompts", op="embed", tokens=16384, vocab=102400, cols=4096, dtype="bf16", pad=0, scale=64.0),
        # the training example's embedding, in fp32 and of an odd width
        dict(name="embed_grad_odd", op="embed_grad", tokens=2048, vocab=512, cols=257, dtype="f32", pad=3, scale=1.0),
        # a training batch over a whole vocabulary: mostly rows without a token
        dict(name="embed_grad_batch", op="embed_grad", tokens=16384, vocab=102400, cols=4096, dtype="bf16", pad=0, scale=64.0),
        # one token through a decoder layer's block: the weights are read once
        dict(name="ffn_token", op="ffn", rows=1, width=4096, inner=14336, dtype="bf16", act="silu", saved="none", pad=0),
        # the same block on a training batch, its pre-activations kept in 8 bits
        dict(name="ffn_batch_mxfp8", op="ffn", rows=8192, width=4096, inner=14336, dtype="bf16", act="silu", saved="mxfp8", pad=0),
        # odd sizes and strides throughout, pre-activations kept as they are
        dict(name="ffn_odd", op="ffn", rows=3001, width=1001, inner=2731, dtype="f16", act="gelu", saved="same", pad=3),
        # the training example's width: launches and latency
        dict(name="ffn_grad_small", op="ffn_grad", rows=2048, width=256, inner=1024, dtype="bf16", act="silu", saved="same",
             x_mxfp8=False, again=False, pad=0),
        # a training batch from 8-bit checkpoints of the input and of both pre-activations, h made again for the next product
        dict(name="ffn_grad_batch_mxfp8", op="ffn_grad", rows=8192, width=4096, inner=14336, dtype="bf16", act="silu", saved="mxfp8",
             x_mxfp8=True, again=True, pad=0),
        # nothing kept but the input: both projections are computed again
        dict(name="ffn_grad_recompute", op="ffn_grad", rows=4096, width=2048, inner=8192, dtype="bf16", act="gelu_tanh", saved="none",
             x_mxfp8=False, again=True, pad=0),
        # a batch's activations to 8 bits
        dict(name="encode_batch", op="encode", rows=16384, cols=4096, dtype="bf16", pad=0),
        # and back, with a row stride of their own
        dict(name="decode_strided", op="decode", rows=6001, cols=2080, dtype="f16", pad=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm, ends included."""
    x = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, x))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "ffn", "ffn", "ffn_grad", "ffn_grad", "encode", "decode"])
    pad = rng.choice([0, 0, 8, rng.randrange(1, 65)])
    if op in ("embed", "embed_grad"):
        cols = _log(rng, 16, 8192)
        return dict(op=op, tokens=min(_log(rng, 1, 65536), (1 << 26) // cols), vocab=min(_log(rng, 16, 131072), (1 << 27) // cols),
                    cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]), pad=pad, scale=rng.choice([1.0, round(cols ** 0.5, 3)]))
    if op in ("encode", "decode"):
        cols = 32 * _log(rng, 1, 512)
        return dict(op=op, rows=min(_log(rng, 1, 65536), (1 << 26) // cols), cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]),
                    pad=pad)
    width, inner = _log(rng, 32, 4096), _log(rng, 32, 14336)
    saved, x_mxfp8 = rng.choice(["none", "same", "mxfp8"]), op == "ffn_grad" and rng.random() < 0.4
    if rng.random() < 0.6:
        width, inner = max(32, width // 8 * 8), max(32, inner // 8 * 8)
    if saved == "mxfp8":
        inner = max(32, inner // 32 * 32)
    if x_mxfp8:
        width = max(32, width // 32 * 32)
    c = dict(op=op, rows=min(_log(rng, 1, 8192), (1 << 38) // (width * inner)), width=width, inner=inner,
             dtype=rng.choice(["bf16", "f16"]), act=rng.choice(ACTS), saved=saved, pad=pad)
    if op == "ffn_grad":
        c.update(x_mxfp8=x_mxfp8, again=rng.random() < 0.5)
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _rows(g, rows, cols, pad, dtype, scale=1.0):
    """rows x cols values with a few wide columns, in rows of cols + pad elements."""
    ld = cols + pad
    col = torch.where(torch.rand(ld, generator=g, device=DEVICE) < 0.01, 8.0, 1.0) * scale
    return (_normal(g, rows, ld) * col).to(DT[dtype])[:, :cols]


def _tokens(g, n, vocab):
    """Token indexes with the low ones frequent (the cube of a uniform number); one in fifty is no token (-1)."""
    u = torch.rand(n, generator=g, device=DEVICE, dtype=torch.float64)
    t = (u ** 3 * vocab).long().clamp_(max=vocab - 1)
    t[torch.rand(n, generator=g, device=DEVICE) < 0.02] = -1
    if n == 1:
        t.clamp_(min=0)
    return t


def _carrier(g, rows, cols):
    """The MXFP8 carrier of normal values: E4M3 codes, exponents of 2 for every 32."""
    x = _normal(g, rows, cols // 32, 32)
    top = x.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top / 448.0)).clamp(-127, 127)
    payload = (x * torch.exp2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, cols)
    return payload.view(torch.uint8), (e + 127).to(torch.uint8).view(rows, cols // 32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    st = {"case": case}
    if own:
        import memory_reduced_muon_gb300 as q
        st["q"] = q
    return {"embed": _prepare_embed, "embed_grad": _prepare_embed_grad, "ffn": _prepare_ffn, "ffn_grad": _prepare_ffn_grad,
            "encode": _prepare_encode, "decode": _prepare_decode}[case["op"]](case, g, st)


def _prepare_embed(c, g, st):
    st["table"] = _rows(g, c["vocab"], c["cols"], c["pad"], c["dtype"], 0.02)
    st["tokens"] = _tokens(g, c["tokens"], c["vocab"])
    st["out"] = torch.empty(c["tokens"], c["cols"], dtype=DT[c["dtype"]], device=DEVICE)
    return st


def _prepare_embed_grad(c, g, st):
    st["dout"] = _rows(g, c["tokens"], c["cols"], c["pad"], c["dtype"], 1e-2)
    st["tokens"] = _tokens(g, c["tokens"], c["vocab"])
    if own:
        st["dtable"] = torch.empty(c["vocab"], c["cols"], dtype=DT[c["dtype"]], device=DEVICE)
        st["ws"] = torch.empty(st["q"].qmuon_embedding_workspace_size(c["tokens"], c["vocab"], c["cols"]), dtype=torch.uint8,
                               device=DEVICE)
    return st


def _weights(c, g, st):
    st["w_gate"] = _rows(g, c["inner"], c["width"], c["pad"], c["dtype"], c["width"] ** -0.5)
    st["w_up"] = _rows(g, c["inner"], c["width"], c["pad"], c["dtype"], c["width"] ** -0.5)


def _prepare_ffn(c, g, st):
    rows, inner, dt = c["rows"], c["inner"], DT[c["dtype"]]
    st["x"] = _rows(g, rows, c["width"], c["pad"], c["dtype"])
    _weights(c, g, st)
    if not own:
        return st
    q = st["q"]
    st["h"] = torch.empty(rows, inner, dtype=dt, device=DEVICE)
    kept = {}
    if c["saved"] == "same":
        kept = {k: torch.empty(rows, inner, dtype=dt, device=DEVICE) for k in ("gate", "up")}
    elif c["saved"] == "mxfp8":
        kept = {k: torch.empty(rows, inner, dtype=torch.uint8, device=DEVICE) for k in ("gate", "up")}
        kept.update({k: torch.empty(rows, inner // 32, dtype=torch.uint8, device=DEVICE) for k in ("gate_scale", "up_scale")})
    st["kept"] = kept
    st["call"] = q.gated_ffn(st["x"], st["w_gate"], st["w_up"], st["h"], rows, c["width"], inner, c["dtype"], act=c["act"],
                             saved=c["saved"], ld_x=st["x"].stride(0), ld_w_gate=st["w_gate"].stride(0),
                             ld_w_up=st["w_up"].stride(0), **kept)
    st["ws"] = torch.empty(q.qmuon_gated_ffn_workspace_size(st["call"]), dtype=torch.uint8, device=DEVICE)
    return st


def _prepare_ffn_grad(c, g, st):
    rows, width, inner, dt = c["rows"], c["width"], c["inner"], DT[c["dtype"]]
    st["dh"] = _rows(g, rows, inner, c["pad"], c["dtype"], 1e-2)
    if c["x_mxfp8"]:
        st["x"], st["x_scale"] = _carrier(g, rows, width)
    else:
        st["x"], st["x_scale"] = _rows(g, rows, width, c["pad"], c["dtype"]), None
    _weights(c, g, st)
    kept = {}
    if c["saved"] == "same":
        kept = {k: _rows(g, rows, inner, c["pad"], c["dtype"]) for k in ("gate", "up")}
    elif c["saved"] == "mxfp8":
        for k in ("gate", "up"):
            kept[k], kept[k + "_scale"] = _carrier(g, rows, inner)
    st.update(kept)
    if not own:
        return st
    q = st["q"]
    st["dx"] = torch.empty(rows, width, dtype=dt, device=DEVICE)
    st["dw_gate"], st["dw_up"] = (torch.empty(inner, width, dtype=dt, device=DEVICE) for _ in range(2))
    st["h"] = torch.empty(rows, inner, dtype=dt, device=DEVICE) if c["again"] else None
    same = {} if c["saved"] != "same" else dict(ld_gate=kept["gate"].stride(0), ld_up=kept["up"].stride(0))
    st["call"] = q.gated_ffn_grad(st["dh"], st["x"], st["w_gate"], st["w_up"], st["dx"], st["dw_gate"], st["dw_up"], rows, width,
                                  inner, c["dtype"], act=c["act"], saved=c["saved"], x_scale=st["x_scale"], h=st["h"],
                                  ld_dh=st["dh"].stride(0), ld_x=st["x"].stride(0), ld_w_gate=st["w_gate"].stride(0),
                                  ld_w_up=st["w_up"].stride(0), **kept, **same)
    st["ws"] = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(st["call"]), dtype=torch.uint8, device=DEVICE)
    return st


def _prepare_encode(c, g, st):
    st["x"] = _rows(g, c["rows"], c["cols"], c["pad"], c["dtype"])
    if own:
        st["payload"] = torch.empty(c["rows"], c["cols"], dtype=torch.uint8, device=DEVICE)
        st["scale"] = torch.empty(c["rows"], c["cols"] // 32, dtype=torch.uint8, device=DEVICE)
    return st


def _prepare_decode(c, g, st):
    st["payload"], st["scale"] = _carrier(g, c["rows"], c["cols"])
    if own:
        st["x"] = torch.empty(c["rows"], c["cols"] + c["pad"], dtype=DT[c["dtype"]], device=DEVICE)[:, :c["cols"]]
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_embed(s):
    c = s["case"]
    s["q"].qmuon_embedding_forward(s["table"], s["tokens"], s["out"], c["tokens"], c["vocab"], c["cols"], c["dtype"], scale=c["scale"],
                                   ld_table=c["cols"] + c["pad"])
    return s["out"]


def _own_embed_grad(s):
    c = s["case"]
    s["q"].qmuon_embedding_backward(s["dout"], s["tokens"], s["dtable"], c["tokens"], c["vocab"], c["cols"], c["dtype"], s["ws"],
                                    scale=c["scale"], ld_dout=c["cols"] + c["pad"])
    return s["dtable"]


def _values(x, scale):
    """What a carrier's bytes stand for."""
    return x.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)


def _own_ffn(s):
    s["q"].qmuon_gated_ffn_forward(s["call"], s["ws"])
    out = {"h": s["h"], **s["kept"]}
    if s["case"]["saved"] == "mxfp8":
        for k in ("gate", "up"):
            out[k], out[k + "_scale"] = _values(out[k], out[k + "_scale"])
    return out


def _own_ffn_grad(s):
    s["q"].qmuon_gated_ffn_backward(s["call"], s["ws"])
    return {k: s[k] for k in ("dx", "dw_gate", "dw_up", "h") if s[k] is not None}


def _own_encode(s):
    c = s["case"]
    s["q"].qmuon_mxfp8_encode(s["x"], s["payload"], s["scale"], c["rows"], c["cols"], c["dtype"], ld_x=c["cols"] + c["pad"])
    payload, scale = _values(s["payload"], s["scale"])
    return {"payload": payload, "scale": scale}


def _own_decode(s):
    c = s["case"]
    s["q"].qmuon_mxfp8_decode(s["payload"], s["scale"], s["x"], c["rows"], c["cols"], c["dtype"], ld_x=c["cols"] + c["pad"])
    return s["x"]


def _plain_embed(s):
    t = s["tokens"]
    rows = s["table"][t.clamp(min=0)].float() * s["case"]["scale"]
    return torch.where((t >= 0)[:, None], rows, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s):
    c, t = s["case"], s["tokens"]
    there = t >= 0
    total = torch.zeros(c["vocab"], c["cols"], device=DEVICE)
    total.index_add_(0, t[there], s["dout"][there].float())
    return (total * c["scale"]).to(s["dout"].dtype)


def _decoded(payload, scale):
    """The fp32 values of a carrier."""
    rows, cols = payload.shape
    x = payload.view(torch.float8_e4m3fn).float().view(rows, cols // 32, 32)
    return torch.ldexp(x, scale.int()[..., None] - 127).view(rows, cols)


def _encoded(x):
    """E4M3 codes and exponent bytes of fp32 rows, to the nearest."""
    rows, cols = x.shape
    x = x.reshape(rows, cols // 32, 32)
    top = x.abs().amax(2, keepdim=True)
    f, e = torch.frexp(top)                          # top = f 2^e, f in [0.5, 1); 448 = 0.875 2^9
    byte = torch.where(top == 0, 127, (e - 9 + 127 + (f > 0.875)).clamp(0, 254))
    payload = torch.ldexp(x, 127 - byte).to(torch.float8_e4m3fn).view(rows, cols)
    return payload, byte.to(torch.uint8).view(rows, -1).view(torch.float8_e8m0fnu)


def _act(name, g):
    """The activation and its derivative in fp32."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * (k * (1.0 + 3 * 0.044715 * g * g))


def _plain_ffn(s):
    c = s["case"]
    dt, x = DT[c["dtype"]], s["x"].float()
    gate, up = x @ s["w_gate"].float().T, x @ s["w_up"].float().T
    out = {"h": (_act(c["act"], gate)[0] * up).to(dt)}
    if c["saved"] == "same":
        out.update(gate=gate.to(dt), up=up.to(dt))
    elif c["saved"] == "mxfp8":
        out["gate"], out["gate_scale"] = _encoded(gate)
        out["up"], out["up_scale"] = _encoded(up)
    return out


def _plain_ffn_grad(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    x = s["x"].float() if s["x_scale"] is None else _decoded(s["x"], s["x_scale"])
    wg, wu, dh = s["w_gate"].float(), s["w_up"].float(), s["dh"].float()
    if c["saved"] == "none":
        gate, up = x @ wg.T, x @ wu.T
    elif c["saved"] == "same":
        gate, up = s["gate"].float(), s["up"].float()
    else:
        gate, up = _decoded(s["gate"], s["gate_scale"]), _decoded(s["up"], s["up_scale"])
    a, slope = _act(c["act"], gate)
    dgate, dup = dh * up * slope, dh * a
    out = {"dx": (dgate @ wg + dup @ wu).to(dt), "dw_gate": (dgate.T @ x).to(dt), "dw_up": (dup.T @ x).to(dt)}
    if c["again"]:
        out["h"] = (a * up).to(dt)
    return out


def _plain_encode(s):
    payload, scale = _encoded(s["x"].float())
    return {"payload": payload, "scale": scale}


def _plain_decode(s):
    return _decoded(s["payload"], s["scale"]).to(DT[s["case"]["dtype"]])


_OWN = {"embed": _own_embed, "embed_grad": _own_embed_grad, "ffn": _own_ffn, "ffn_grad": _own_ffn_grad, "encode": _own_encode,
        "decode": _own_decode}
_PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "ffn": _plain_ffn, "ffn_grad": _plain_ffn_grad,
          "encode": _plain_encode, "decode": _plain_decode}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _distinct(n, vocab):
    """Expected number of different tokens among n of `_tokens`."""
    edge = np.cbrt(np.arange(vocab + 1) / vocab)
    return float(np.sum(-np.expm1(0.98 * n * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12)))))


def work(case):
    c, op = case, case["op"]
    size = SIZE[c["dtype"]]
    if op == "embed":
        n = c["tokens"] * c["cols"]
        return {"bytes": 8 * c["tokens"] + int(_distinct(c["tokens"], c["vocab"]) * c["cols"] * size) + n * size, "flops": n}
    if op == "embed_grad":
        n = c["tokens"] * c["cols"]
        return {"bytes": 8 * c["tokens"] + n * size + c["vocab"] * c["cols"] * size, "flops": n}
    if op in ("encode", "decode"):
        n = c["rows"] * c["cols"]
        return {"bytes": n * size + n + n // 32, "flops": 2 * n}
    rows, width, inner = c["rows"], c["width"], c["inner"]
    kept = {"none": 0, "same": 2 * size, "mxfp8": 2 + 2 / 32}[c["saved"]]
    weights = 2 * inner * width * size
    if op == "ffn":
        return {"bytes": int(rows * width * size + weights + rows * inner * (size + kept)), "flops": 4 * rows * width * inner}
    x = rows * width * (1 + 1 / 32 if c["x_mxfp8"] else size)
    move = x + 2 * weights + rows * width * size + rows * inner * (size * (2 if c["again"] else 1) + kept)
    return {"bytes": int(move), "flops": (12 if c["saved"] == "none" else 8) * rows * width * inner}


# --------------------------------------------------------------------------
# the definitions in fp64
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "ffn": _exact_ffn, "ffn_grad": _exact_ffn_grad,
            "encode": _exact_encode, "decode": _exact_decode}[case["op"]](case, s)


def _exact_embed(c, s):
    out = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device=DEVICE)
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    out[at] = s["table"][s["tokens"][at]].double() * c["scale"]
    return out


def _exact_embed_grad(c, s):
    out = torch.zeros(c["vocab"], c["cols"], dtype=torch.float64, device=DEVICE)
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    return out.index_put_((s["tokens"][at],), s["dout"][at].double() * c["scale"], accumulate=True)


def _exact_values(payload, scale):
    codes = payload.view(torch.float8_e4m3fn).double().unflatten(1, (-1, 32))
    return (codes * torch.exp2(scale.double() - 127).unsqueeze(2)).flatten(1)


def _exact_codes(x):
    """The nearest E4M3 values (ties to even; 3 mantissa bits, exponents from -6 up, largest 448) under the smallest power
    of two that leaves the largest of 32 within 448, and these powers."""
    x = x.unflatten(1, (-1, 32))
    top = x.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)       # a logarithm that is rounded up from a whole number
    e = torch.where(top > 0, e, 0.0).clamp(-127, 127)
    x = x * torch.exp2(-e)
    grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / grid) * grid).clamp_(-448, 448).flatten(1), torch.exp2(e).flatten(1)


def _exact_act(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if name == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, torch.addcmul(cdf, g, torch.exp(g * g / -2), value=(2 * math.pi) ** -0.5)
    w = (8 / math.pi) ** 0.5
    s = torch.sigmoid(w * g + 0.044715 * w * g ** 3)      # (1 + tanh z) / 2 = sigmoid(2 z)
    return g * s, s + g * s * (1 - s) * (w + 3 * 0.044715 * w * g ** 2)


def _exact_ffn(c, s):
    x = s["x"].double()
    gate, up = torch.mm(x, s["w_gate"].double().t()), torch.mm(x, s["w_up"].double().t())
    out = {"h": _exact_act(c["act"], gate)[0].mul_(up)}
    if c["saved"] == "same":
        out.update(gate=gate, up=up)
    elif c["saved"] == "mxfp8":
        out["gate"], out["gate_scale"] = _exact_codes(gate)
        out["up"], out["up_scale"] = _exact_codes(up)
    return out


def _exact_ffn_grad(c, s):
    x = _exact_values(s["x"], s["x_scale"]) if c["x_mxfp8"] else s["x"].double()
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    if c["saved"] == "none":
        gate, up = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    elif c["saved"] == "same":
        gate, up = s["gate"].double(), s["up"].double()
    else:
        gate, up = _exact_values(s["gate"], s["gate_scale"]), _exact_values(s["up"], s["up_scale"])
    a, slope = _exact_act(c["act"], gate)
    h = a * up if c["again"] else None
    dh = s["dh"].double()
    dgate, dup = up.mul_(slope).mul_(dh), a.mul_(dh)
    out = {"dx": torch.mm(dgate, wg).addmm_(dup, wu), "dw_gate": torch.mm(dgate.t(), x), "dw_up": torch.mm(dup.t(), x)}
    return {**out, "h": h} if c["again"] else out


def _exact_encode(c, s):
    payload, scale = _exact_codes(s["x"].double())
    return {"payload": payload, "scale": scale}


def _exact_decode(c, s):
    return _exact_values(s["payload"], s["scale"])
