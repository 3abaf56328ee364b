"""Token embedding, gated feed-forward block and 8-bit activation checkpoints --
CPU oracle (test infrastructure only).

The definitions that the library's header states, in fp64; the checkpoint
codec, whose results are compared bit for bit, takes fp32 values.
"""

from __future__ import annotations

import math

import numpy as np

from . import carrier

F64 = np.float64


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embedding64(table, tokens, scale: float = 1.0):
    """Rows of `table` times `scale`; zeros for a token outside."""
    table, tokens = np.asarray(table, F64), np.asarray(tokens)
    out = np.zeros((tokens.size, table.shape[1]))
    for t, v in enumerate(tokens):
        if 0 <= v < table.shape[0]:
            out[t] = table[v] * scale
    return out


def embedding_grad64(dout, tokens, vocab: int, scale: float = 1.0):
    """(the table's gradient, the sum of its terms' magnitudes, the number of its terms)."""
    dout, tokens = np.asarray(dout, F64), np.asarray(tokens)
    grad, mag, count = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros(vocab, np.int64)
    for t, v in enumerate(tokens):
        if 0 <= v < vocab:
            grad[v] += dout[t]
            mag[v] += np.abs(dout[t])
            count[v] += 1
    return grad * scale, mag * abs(scale), count


# --------------------------------------------------------------------------
# gated feed-forward block
# --------------------------------------------------------------------------

def act64(name: str, g):
    """(act(g), act'(g))."""
    g = np.asarray(g, F64)
    with np.errstate(over="ignore"):
        if name == "silu":
            s = 1.0 / (1.0 + np.exp(-g))
            return g * s, s + g * s * (1.0 - s)
        if name == "gelu":
            cdf = 0.5 * np.vectorize(math.erfc, otypes=[F64])(-g / math.sqrt(2.0))
            return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        if name == "gelu_tanh":
            k = math.sqrt(2.0 / math.pi)
            t = np.tanh(k * (g + 0.044715 * g ** 3))
            return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)
    raise ValueError(name)


def gated_ffn64(x, w_gate, w_up, act: str):
    """(h, gate, up)."""
    x = np.asarray(x, F64)
    gate, up = x @ np.asarray(w_gate, F64).T, x @ np.asarray(w_up, F64).T
    return act64(act, gate)[0] * up, gate, up


def gated_slopes64(dh, gate, up, act: str):
    """(dgate, dup, h) of given gate and up."""
    dh, gate, up = (np.asarray(v, F64) for v in (dh, gate, up))
    a, slope = act64(act, gate)
    return dh * up * slope, dh * a, a * up


def gated_products64(dgate, dup, x, w_gate, w_up):
    """(dx, dw_gate, dw_up) of given dgate and dup."""
    dgate, dup, x = (np.asarray(v, F64) for v in (dgate, dup, x))
    return dgate @ np.asarray(w_gate, F64) + dup @ np.asarray(w_up, F64), dgate.T @ x, dup.T @ x


# --------------------------------------------------------------------------
# 8-bit checkpoints
# --------------------------------------------------------------------------

def encode(x: np.ndarray):
    """(payload, scale bytes) of fp32 rows: the carrier's codec."""
    return carrier.encode_rows(np.asarray(x, np.float32))


def decode64(payload, scale):
    """The carrier's values in fp64."""
    rows, cols = payload.shape
    codes = carrier.e4m3_decode(np.asarray(payload).reshape(-1)).astype(F64).reshape(rows, cols // 32, 32)
    return (codes * 2.0 ** (np.asarray(scale, F64) - 127.0)[..., None]).reshape(rows, cols)
