"""Rotary positions and cross attention, from the definitions in ``include/bsa.h``.

Angles are exact: the fraction of a turn is taken in Python integers.  ``rotate_f32`` rounds every product and sum to
float32 as the definition says; ``rotate`` is the same in float64."""

import math

import numpy as np

from .attention import softmax_attention


def rotary_table(positions, turns, axis=None, factor=1.0):
    """positions [T] or [T, axes], turns [P] (2^-64 turns a position) -> cos, sin [T, P] in float64."""
    positions = np.asarray(positions)
    positions = positions.reshape(positions.shape[0], -1)
    cos, sin = np.zeros((positions.shape[0], len(turns))), np.zeros((positions.shape[0], len(turns)))
    for t in range(positions.shape[0]):
        for i, f in enumerate(turns):
            frac = (int(positions[t, axis[i] if axis is not None else 0]) * int(f)) % (1 << 64)
            if frac >= 1 << 63:
                frac -= 1 << 64  # half a turn to either side: the float64 angle then loses nothing near 0
            angle = 2 * math.pi * (frac / 2.0 ** 64)
            cos[t, i], sin[t, i] = factor * math.cos(angle), factor * math.sin(angle)
    return cos, sin


def _halves(x, P, interleaved):
    return (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])


def _join(a, b, rest, interleaved):
    turned = np.stack([a, b], -1).reshape(a.shape[:-1] + (-1,)) if interleaved else np.concatenate([a, b], -1)
    return np.concatenate([turned, rest], -1)


def rms_norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, cos, sin, interleaved=False, transpose=False):
    """Rows x [T, heads, D] by tables [T, P], in float64."""
    x, P = np.asarray(x, dtype=np.float64), cos.shape[-1]
    c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None] * (-1.0 if transpose else 1.0)
    a, b = _halves(x, P, interleaved)
    return _join(a * c - b * s, b * c + a * s, x[..., 2 * P:], interleaved)


def rotate_f32(x, cos, sin, interleaved=False, transpose=False):
    """The same with every product and sum rounded to float32."""
    x, P = np.asarray(x, dtype=np.float32), cos.shape[-1]
    c, s = np.asarray(cos, np.float32)[:, None], np.asarray(sin, np.float32)[:, None]
    s = -s if transpose else s
    a, b = _halves(x, P, interleaved)
    with np.errstate(all="ignore"):
        return _join(a * c - b * s, b * c + a * s, x[..., 2 * P:], interleaved)


def cross_attention(q, k, v, scale):
    """Rows q [n, HQ, D] over the states k, v [m, H, D]: (o [n, HQ, D], lse [n, HQ])."""
    n, HQ, D = q.shape
    o, lse = np.zeros((n, HQ, D)), np.full((n, HQ), -np.inf)
    for hq in range(HQ):
        h = hq * k.shape[1] // HQ
        if n and k.shape[0]:
            o[:, hq], lse[:, hq] = softmax_attention(q[:, hq], k[:, h], v[:, h], scale)
    return o, lse
