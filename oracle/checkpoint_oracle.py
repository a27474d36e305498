"""Plain fp64 numpy definitions of activation checkpoints in 8 bits and of the steps that read them: test
infrastructure, written from the formulas and independent of the HIP path."""
from __future__ import annotations

import numpy as np

from .router_oracle import U

GROUP = 128


def groups(width):
    return -(-width // GROUP)


def bf16_at_least(x):
    """The smallest bf16 number >= x, for x >= 0 within its normal range."""
    m, e = np.frexp(np.asarray(x, np.float64))  # m in [0.5, 1)
    return np.ldexp(np.ceil(m * 256.0), e - 8)


def _split(x, parts):
    """[n, parts * w] as [n, parts, groups, 128], zeros behind w."""
    n, w = x.shape[0], x.shape[1] // parts
    y = np.zeros((n, parts, groups(w) * GROUP))
    y[:, :, :w] = np.asarray(x, np.float64).reshape(n, parts, w)
    return y.reshape(n, parts, groups(w), GROUP)


def _join(y, width):
    n, parts = y.shape[:2]
    return y.reshape(n, parts, -1)[:, :, :width // parts].reshape(n, width)


def checkpoint(x, parts):
    """(q [n, width], scale [n, parts, groups]) in fp64; exact for f32 and bf16 values."""
    y = _split(x, parts)
    bad = ~np.isfinite(y).all(3)
    z = np.where(bad[..., None], 0.0, y)
    scale = np.maximum(bf16_at_least(np.abs(z).max(3) / 127.0), 2.0 ** -126)
    q = np.rint(z / scale[..., None])  # a quotient within 2^-53 of a half is one: x and s have 32 bits together
    return _join(q, x.shape[1]), np.where(bad, np.nan, scale)


def values(q, scale):
    return _join(_split(q, scale.shape[1]) * np.asarray(scale, np.float64)[..., None], q.shape[1])


def phi(h, swiglu):
    """(phi, err): err bounds an fp32 evaluation from the same h. exp(-g) has the rounding of g log2 e, a relative |g| U,
    of which sigmoid keeps the part 1 - sigmoid(g); exponential, sum, reciprocal and two products stay under 8 U. A sigmoid
    below 2^-126 (g under -87.3) is a subnormal number, which the reciprocal gives as 0: |g| sigmoid(g) is at most
    87.4 * 2^-126 = 2^-119.55 there, as it falls with g."""
    if not swiglu:
        return h, np.zeros_like(h)
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    with np.errstate(over="ignore"):
        sg = 1.0 / (1.0 + np.exp(-g))
    p = g * sg * u
    return p, np.abs(p) * ((1 - sg) * np.abs(g) + 8) * U + np.abs(u) * 2.0 ** -119.5


def score(G, q, scale, alpha, tok, swiglu):
    """(R, err) with G in fp64."""
    p, e = phi(values(q, scale), swiglu)
    a = np.asarray(alpha, np.float64)
    f = a * a * (G * G).sum(1)[tok]
    R = f * (p * p).sum(1)
    return R, f * (2 * np.abs(p) * e).sum(1) * (1 + 2.0 ** -20) + R * 2 * U + 1e-44


def compact(sel, q, scale, alpha, swiglu, bf16):
    """(PhiW, err) of the rows sel; rows outside the pairs are zeros."""
    ok = (sel >= 0) & (sel < len(q))
    at = np.where(ok, sel, 0)
    p, e = phi(values(q[at], np.asarray(scale, np.float64)[at]), swiglu)
    a = np.where(ok, np.asarray(alpha, np.float64)[at], 0.0)[:, None]
    w = np.where(ok[:, None], a * p, 0.0)
    err = np.abs(a) * e + np.abs(w) * U
    return w, np.where(ok[:, None], err + (np.abs(w) * 2.0 ** -8 + 2.0 ** -134 if bf16 else 1e-44), 0.0)
