"""Plain fp64 CPU forms of the operators around the attention: rotary positions, the gated feed-forward block and the
global gradient norm with clipping. Written from the definitions; nothing on the product path imports this."""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(n, theta=10000.0, scaling="none", factor=1.0, trained_len=4096.0):
    """Radians per position of the n / 2 pairs of one axis."""
    out = []
    for j in range(n // 2):
        base = theta * factor ** (n / (n - 2.0)) if scaling == "ntk" and n > 2 else theta
        f = base ** (-2.0 * j / n)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            def index(turns):  # the pair that turns that often over the trained length
                return n * math.log(trained_len / (2 * math.pi * turns)) / (2 * math.log(theta))
            low, high = max(math.floor(index(32)), 0), min(math.ceil(index(1)), n - 1)
            t = min(max((j - low) / max(high - low, 0.001), 0.0), 1.0)
            f = (1 - t) * f + t * f / factor
        out.append(f)
    return np.array(out)


def rope_angles(axis_dims, grid=None, positions=None, n=None, pos_scale=None, pos_offset=None, **freq):
    """[tokens, pairs] radians."""
    k = len(axis_dims)
    if positions is not None:
        p = np.asarray(positions, dtype=np.float64).reshape(-1, k)
    elif k == 3:
        p = np.stack(np.meshgrid(*[np.arange(g, dtype=np.float64) for g in grid], indexing="ij"), -1).reshape(-1, 3)
    else:
        p = np.arange(n, dtype=np.float64)[:, None]
    scale, offset = pos_scale or (1.0,) * k, pos_offset or (0.0,) * k
    return np.concatenate([(offset[a] + p[:, a:a + 1] * scale[a]) * rope_frequencies(axis_dims[a], **freq)[None]
                           for a in range(k)], axis=1)


def rope(x, angles, layout, magnitude=1.0, transposed=False):
    """x [tokens, heads, d] rotated, fp64."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    pairs = angles.shape[1]
    c, s = magnitude * np.cos(angles)[:, None], magnitude * np.sin(angles)[:, None]
    if transposed:
        s = -s
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + pairs)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


# ------------------------------------------------------------------ gated feed-forward
def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def activation(act, g):
    if act == "silu":
        return g / (1 + np.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + _erf(g / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return np.maximum(g, 0)


def activation_slope(act, g):
    if act == "silu":
        s = 1 / (1 + np.exp(-g))
        return s + g * s * (1 - s)
    if act == "gelu":
        return 0.5 * (1 + _erf(g / math.sqrt(2))) + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    return (g > 0).astype(np.float64)


def gated_ffn_fwd(x, wg, wu, wd, act):
    """(y, g, u)."""
    g, u = x @ wg.T, x @ wu.T
    return (activation(act, g) * u) @ wd.T, g, u


def gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act):
    """(dx, dwg, dwu, dwd) at the given projections g, u."""
    a, dh = activation(act, g), dy @ wd
    dg, du = dh * u * activation_slope(act, g), dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)


# ------------------------------------------------------------------ gradient norm
def grad_norm(grads, ord=2):
    if ord == 2:
        return math.sqrt(math.fsum(float(np.sum(np.square(g.astype(np.longdouble)))) for g in grads))
    return max((float(np.max(np.abs(g))) for g in grads if g.size), default=0.0)


def clip_factor(norm, max_norm, eps=1e-6):
    return min(1.0, max_norm / (norm + eps))
