"""Gradient clipping, AdamW and the RMS norm -- CPU oracle (test infrastructure only).

The pages name AdamW as Muon's companion for the parameters that are not
matrices and give no formulas; these are the definitions the library's header
states.  Functions ending in ``64`` evaluate them in fp64.  The others
evaluate the header's operation order in fp32, one rounding per operation, so
that 8-bit states can be compared bit for bit:

* 8-bit AdamW states: E4M3 codes of the first moment ``m`` and of the square
  root ``r`` of the second, one fp32 maximum per 256 elements;
  ``x = code * (max / 448)``; new codes from ``x * min(448 / max, FLT_MAX)``,
  at least 1 for a root above zero;
* stochastic requantisation: magnitudes are cut to the 3-bit grid after 16
  random bits are added below it (``oracle.rng`` words: the low half for m, the
  high half for r);
* a NaN lane is ignored by the maximum and keeps a NaN code.
"""

from __future__ import annotations

import math

import numpy as np

from . import carrier, rng

F32 = np.float32
BLOCK = 256
FLT_MAX = np.finfo(np.float32).max


# --------------------------------------------------------------------------
# clipping
# --------------------------------------------------------------------------

def clip64(grads, max_norm: float):
    """(norm, coefficient) of a list of arrays; the coefficient is NaN where the norm is not finite."""
    norm = math.sqrt(math.fsum(float(np.sum(np.square(np.asarray(g, dtype=np.float64)))) for g in grads))
    return norm, (min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else math.nan)


# --------------------------------------------------------------------------
# AdamW
# --------------------------------------------------------------------------

def adamw64(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay=0.0, scale=1.0):
    """New (p, m, v) in fp64."""
    p, g, m, v = (np.asarray(x, dtype=np.float64) for x in (p, g, m, v))
    g = g * scale
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    u = (m / (1.0 - beta1 ** t)) / (np.sqrt(v / (1.0 - beta2 ** t)) + eps)
    return p - lr * weight_decay * p - lr * u, m, v


def block_max(x: np.ndarray) -> np.ndarray:
    """max |x| per 256 elements, NaN lanes ignored."""
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, dtype=x.dtype)
    pad[:n] = np.abs(x)
    pad[np.isnan(pad)] = 0
    return pad.reshape(-1, BLOCK).max(1)


def spread(per_block: np.ndarray, n: int) -> np.ndarray:
    return np.repeat(per_block, BLOCK)[:n]


def e4m3_stochastic(x: np.ndarray, u16: np.ndarray) -> np.ndarray:
    """E4M3 codes of fp32 x: |x| on the grid of its binade (2^-9 below 2^-6), rounded up where the fraction of a step
    plus u16 / 65536 reaches 1; saturating; NaN to 0x7F."""
    a = np.abs(x.astype(np.float64))
    with np.errstate(invalid="ignore"):
        e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
        step = 2.0 ** (np.where(np.isfinite(e), e, 0) - 3)
        k = np.floor(np.where(np.isfinite(a), a, 0) / step + u16.astype(np.float64) / 65536)
        mag = np.minimum(k * step, 448.0).astype(F32)
    code = carrier.e4m3_encode(mag).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    code = np.where(np.isinf(x), 0x7E | (np.signbit(x).astype(np.uint8) << 7), code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def root_codes(codes: np.ndarray, scaled: np.ndarray) -> np.ndarray:
    """Codes of the scaled roots: 1 instead of 0 where the root is above zero (and its block's maximum finite)."""
    return np.where((scaled > 0) & (codes == 0), np.uint8(1), codes)


def adamw_e4m3(p, g, m, v, m_max, v_max, t, lr, beta1, beta2, eps, weight_decay=0.0, lr_scale=1.0, scale=1.0,
               seed=None, tensor_index=0):
    """New (p, m codes, v codes, m_max, v_max) in the header's fp32 order; ``seed``: stochastic requantisation."""
    n = p.size
    with np.errstate(all="ignore"):
        g = g.astype(F32) * F32(scale)
        m0 = carrier.e4m3_decode(m).astype(F32) * spread(m_max / F32(448), n)
        r0 = carrier.e4m3_decode(v).astype(F32) * spread(v_max / F32(448), n)
        m1 = m0 * F32(beta1) + g * F32(1.0 - beta1)
        v1 = (r0 * r0) * F32(beta2) + (g * g) * F32(1.0 - beta2)
        r1 = np.sqrt(v1)
        u = m1 / (r1 * F32(1.0 / math.sqrt(1.0 - beta2 ** t)) + F32(eps))
        lr_t = F32(lr) * F32(lr_scale)
        p1 = p * (F32(1) - lr_t * F32(weight_decay)) - (lr_t * F32(1.0 / (1.0 - beta1 ** t))) * u
        mm, vm = block_max(m1), block_max(r1)
        mx = m1 * spread(np.minimum(F32(448) / mm, FLT_MAX), n)
        vx = r1 * spread(np.minimum(F32(448) / vm, FLT_MAX), n)
        if seed is None:
            return p1, carrier.e4m3_encode(mx), root_codes(carrier.e4m3_encode(vx), vx), mm, vm
        j = np.arange((n + 3) // 4, dtype=np.uint64)
        ctr = np.stack([j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, tensor_index),
                        np.full_like(j, t & 0xFFFFFFFF)], 1)
        w = rng.philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)[:n]
        return p1, e4m3_stochastic(mx, w & 0xFFFF), root_codes(e4m3_stochastic(vx, w >> 16), vx), mm, vm


# --------------------------------------------------------------------------
# RMS norm
# --------------------------------------------------------------------------

def rmsnorm64(x, gain, eps, residual=None):
    """(h, y)."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    return h, h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(gain, dtype=np.float64)


def rmsnorm_grad64(dy, h, gain, eps, dsum=None):
    """(dx, dgain) of sum(dy * y(h)) + sum(dsum * h)."""
    dy, h, gain = (np.asarray(a, dtype=np.float64) for a in (dy, h, gain))
    inv = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n, a = h * inv, dy * gain
    dx = inv * (a - n * np.mean(a * n, axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, dtype=np.float64)
    return dx, np.sum(dy * n, axis=0)
