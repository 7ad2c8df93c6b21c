"""Plain fp64 forms of what stands around the experts: residual add and layer
norm with its gradient, the experts' FFN on 8-bit integers, the gradient norm and
clipping.

Written from the formulas, in NumPy, sharing no code with the GPU path. Where the
operator's definition rounds on the way (a sum held in the rows' type, codes and
scales), the caller passes the rounding as a function or the codes themselves.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, weight, bias, eps, residual=None, hold=None):
    """(y, s, mean, rstd) in fp64; hold rounds s = x + residual to the rows' type."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + residual
        if hold is not None:
            s = hold(s)
    mean = s.mean(axis=1)
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c ** 2).mean(axis=1) + eps)
    y = c * rstd[:, None] * weight
    if bias is not None:
        y = y + bias
    return y, s, mean, rstd


def layer_norm_backward(d_y, s, weight, mean, rstd, d_s=None):
    """(d_x, d_weight, d_bias) in fp64 for the given statistics."""
    h = (s - mean[:, None]) * rstd[:, None]
    g = d_y * weight
    d_x = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - h * (g * h).mean(axis=1, keepdims=True))
    if d_s is not None:
        d_x = d_x + d_s
    return d_x, (d_y * h).sum(axis=0), d_y.sum(axis=0)


def quantize(a):
    """Codes and scales along the last axis of an fp32 array, step by step in fp32
    as the operator defines them: scale = max(max|a| / 127, 2^-126), q = rint(a *
    (1 / scale)); a row with an infinity or NaN has scale NaN and codes 0."""
    a = np.asarray(a, dtype=np.float32)
    finite = np.isfinite(a).all(axis=-1)
    top = np.abs(np.where(finite[..., None], a, np.float32(0))).max(axis=-1)
    scale = np.maximum(top / np.float32(127), np.float32(2.0 ** -126)).astype(np.float32)
    inv = np.float32(1) / scale
    q = np.rint(np.where(finite[..., None], a, np.float32(0)) * inv[..., None]).astype(np.int8)
    return q, np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def kblocks(q):
    """Codes [..., R, K] in K-blocks of 64: [..., ceil(K / 64), R, 64], zero past K."""
    k = q.shape[-1]
    pad = [(0, 0)] * (q.ndim - 1) + [(0, -k % 64)]
    p = np.pad(q, pad)
    return np.ascontiguousarray(np.moveaxis(p.reshape(*p.shape[:-1], p.shape[-1] // 64, 64), -2, -3))


def from_kblocks(b, k):
    """The inverse of kblocks for K = k columns."""
    m = np.moveaxis(b, -3, -2)
    return m.reshape(*m.shape[:-2], m.shape[-2] * 64)[..., :k]


def int8_product(q, scale, wq, wscale):
    """(q [R, K] @ wq [N, K]^T) * scale [R] * wscale [N]: exact integer sums, then fp64."""
    acc = q.astype(np.float64) @ wq.astype(np.float64).T  # integers below 2^53: exact
    return acc * scale.astype(np.float64)[:, None] * wscale.astype(np.float64)[None, :]


def swiglu(gu):
    """silu(gate) * up of [R, 2 * d_ff]."""
    g, u = np.split(gu, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def grad_norm(grads):
    """2-norm over a list of fp64 arrays."""
    return float(np.sqrt(sum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads)))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))
