"""Plain forms of routing by scores with its gradient, RMS norm with its gradient and
the AdamW step, in fp64.

Written from the formulas, in NumPy, sharing no code with the GPU path. Where the
operator's definition rounds on the way (choice values held in fp32, states held in
8 bits), the rounding is part of the plain form.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------ routing

def sigmoid(x):
    """1 / (1 + e^-x) in fp64; an e^-x that overflows gives 0."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def softmax(x):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        p = np.exp(x - x.max(axis=-1, keepdims=True))
    return p / p.sum(axis=-1, keepdims=True)


def _place(v):
    """Sort key of one value, first things first: numbers from the largest down, then NaN."""
    return (1, 0.0) if np.isnan(v) else (0, -float(v))


def choice_values(logits, score, bias=None, groups=1, group_top=2):
    """What the choice goes by, fp32 [T, E]: the logits, or round32(score + bias), -infinity (unless
    that is a NaN) where the logit is."""
    logits = np.asarray(logits, dtype=np.float32)
    if bias is None and (groups == 1 or group_top == 1):
        return logits
    s = sigmoid(logits) if score == "sigmoid" else softmax(logits)
    if bias is not None:
        s = s + np.asarray(bias, dtype=np.float64)
    c = s.astype(np.float32)
    return np.where(np.isneginf(logits) & ~np.isnan(c), np.float32(-np.inf), c)


def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True,
                  scale=1.0):
    """(idx [T, k], w [T, k] fp64), token by token."""
    logits = np.asarray(logits, dtype=np.float32)
    T, E = logits.shape
    c, size = choice_values(logits, score, bias, groups, group_top), E // groups
    idx = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        stay = range(groups)
        if top_groups < groups:
            value = []
            for g in range(groups):
                best = sorted(c[t, g * size:(g + 1) * size], key=_place)
                with np.errstate(invalid="ignore", over="ignore"):
                    v = best[0] + best[1] if group_top == 2 and size > 1 else best[0]  # fp32
                # sums of -infinity go by the largest
                value.append((*_place(v), *(_place(best[0]) if v == -np.inf else (0, 0.0))))
            stay = sorted(range(groups), key=lambda g: (*value[g], g))[:top_groups]
        from_ = [e for g in stay for e in range(g * size, (g + 1) * size)]
        idx[t] = sorted(from_, key=lambda e: (*_place(c[t, e]), e))[:k]
        x = logits[t, idx[t]]
        if score == "sigmoid":
            s = sigmoid(x)
            w[t] = s / (s.sum() + 1e-20) if renormalize else s
        else:
            w[t] = softmax(x) if renormalize else softmax(logits[t])[idx[t]]
    return idx, scale * w


def route_experts_backward(logits, idx, d_w, score="softmax", renormalize=True, scale=1.0):
    """d_logits [T, E] fp64: the chain rule through the weights of the given ids (those
    outside [0, E) are left out)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        keep = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        e, u = idx[t, keep], scale * np.asarray(d_w, dtype=np.float64)[t, keep]
        x = logits[t, e]
        if score == "sigmoid":
            s = sigmoid(x)
            slope = s * sigmoid(-x)
            if renormalize:
                S = s.sum() + 1e-20
                out[t, e] = [sum(u[j] * ((i == j) / S - s[j] / S ** 2) for j in range(len(e))) * slope[i]
                             for i in range(len(e))]
            else:
                out[t, e] = u * slope
        elif renormalize:
            if len(e):
                q = softmax(x)
                out[t, e] = q * (u - (u * q).sum())
        else:
            p = softmax(logits[t])
            g = np.zeros(E)
            g[e] = u
            out[t] = p * (g - (g * p).sum())
    return out


# ----------------------------------------------------------------------- RMS norm

def rms_norm(x, weight, eps, residual=None, hold=None):
    """(y, s, rstd) in fp64; hold rounds s = x + residual to the rows' type."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + residual
        if hold is not None:
            s = hold(s)
    rstd = 1.0 / np.sqrt((s ** 2).mean(axis=1) + eps)
    return s * rstd[:, None] * weight, s, rstd


def rms_norm_backward(d_y, s, weight, rstd, d_s=None):
    """(d_x, d_weight) in fp64 for the given statistic."""
    h = s * rstd[:, None]
    g = d_y * weight
    d_x = rstd[:, None] * (g - h * (g * h).mean(axis=1, keepdims=True))
    if d_s is not None:
        d_x = d_x + d_s
    return d_x, (d_y * h).sum(axis=0)


# -------------------------------------------------------------------------- AdamW

def _e4m3_values():
    """The finite values of the codes 0..126 (sign 0): 4 exponent bits with bias 7, 3 bits of
    significand, the exponent 0 without the leading one."""
    out = []
    for code in range(127):
        e, f = code >> 3, code & 7
        out.append(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = _e4m3_values()
BLOCK = 128


def from_e4m3(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    with np.errstate(invalid="ignore"):
        return np.where(codes & 0x7F == 0x7F, np.nan, E4M3[np.minimum(codes & 0x7F, 126)]) * np.where(codes & 0x80, -1.0, 1.0)


def to_e4m3(a):
    """The nearest code (ties to the even one) of values of at most 448."""
    a = np.asarray(a, dtype=np.float64)
    mag = np.minimum(np.abs(a), 448.0)
    hi = np.clip(np.searchsorted(E4M3, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - mag, mag - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(a), 0x80, 0)).astype(np.uint8)


def mix(h):
    """The finaliser of MurmurHash3, of uint32 arrays."""
    h = np.asarray(h, dtype=np.uint32)
    with np.errstate(over="ignore"):
        h = (h ^ h >> np.uint32(16)) * np.uint32(0x85EBCA6B)
        h = (h ^ h >> np.uint32(13)) * np.uint32(0xC2B2AE35)
    return h ^ h >> np.uint32(16)


def dither_bits(index, step):
    """32 random bits for each element of a tensor (int64 indices) in a step: the lower 16 for the first
    state, the upper for the second."""
    index = np.asarray(index, dtype=np.uint64)
    low, high = (index & np.uint64(0xFFFFFFFF)).astype(np.uint32), (index >> np.uint64(32)).astype(np.uint32)
    key = mix(np.uint32(step & 0xFFFFFFFF) ^ mix(np.uint32(step >> 32)))
    with np.errstate(over="ignore"):
        return mix(low ^ mix(high + key))


def to_e4m3_dithered(a, bits):
    """One of the two codes around each fp32 value of at most 448, by 16 random bits: up where the share
    of the way there and the bits (as a fraction, half a unit more) add up to one."""
    mag, bits = np.abs(np.asarray(a, dtype=np.float32)), np.asarray(bits, dtype=np.uint32)
    # below 2^-6 codes are 2^-9 apart, as they are for another 2^-6 on top
    shift = np.where(mag < np.float32(2.0 ** -6), np.float32(2.0 ** -6), np.float32(0))
    up = (((mag + shift).view(np.uint32) + (bits << np.uint32(4) | np.uint32(8))) & np.uint32(0xFFF00000)).view(np.float32) - shift
    return to_e4m3(np.copysign(np.minimum(up, np.float32(448)), a))


def encode_state(a, root=False, bits=None):
    """Codes and scales of an fp32 array, step by step in fp32 as the operator defines
    them; a root above 0 has at least the code 1. bits: dither_bits of its elements."""
    a = np.asarray(a, dtype=np.float32)
    n = a.size
    b = np.pad(a.reshape(-1), (0, -n % BLOCK)).reshape(-1, BLOCK)
    finite = np.isfinite(b).all(axis=1)
    safe = np.where(finite[:, None], b, np.float32(0))
    scale = np.maximum(np.abs(safe).max(axis=1) * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126))
    scaled = safe * (np.float32(1) / scale)[:, None]
    if bits is None:
        codes = to_e4m3(scaled)
    else:
        half = np.asarray(bits).reshape(-1) >> np.uint32(16) if root else np.asarray(bits).reshape(-1) & np.uint32(0xFFFF)
        codes = to_e4m3_dithered(scaled, np.pad(half, (0, -n % BLOCK)).reshape(-1, BLOCK))
    codes = np.where(finite[:, None], codes, 0).astype(np.uint8)
    if root:
        codes = np.where((safe > 0) & (codes == 0), 1, codes).astype(np.uint8)
    return codes.reshape(-1)[:n], np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def decode_state(codes, scale):
    """What codes and scales stand for, in fp64."""
    n = codes.size
    return from_e4m3(codes.reshape(-1)) * np.repeat(scale.astype(np.float64), BLOCK)[:n]


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, coef=1.0):
    """(p, m, v) after the step, in fp64."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    b1, b2 = betas
    g = g * coef
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    hat_m, hat_v = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * weight_decay * p - lr * hat_m / (np.sqrt(hat_v) + eps), m, v


def adamw_states32(g, m, root, betas, coef=1.0):
    """(m, sqrt(v)) after the step, every product and sum rounded to fp32, from states
    held in 8 bits (fp32 m and root): what their new codes are taken from."""
    f = np.float32
    b1, b2 = betas
    with np.errstate(over="ignore", invalid="ignore"):
        g = np.asarray(g, dtype=f) * f(coef)
        m = np.asarray(m, dtype=f) * f(b1) + g * f(1 - b1)
        root = np.asarray(root, dtype=f)
        v = root * root * f(b2) + g * g * f(1 - b2)
        return m, np.sqrt(v)
