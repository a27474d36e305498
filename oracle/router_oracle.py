"""Plain fp64 numpy definitions of the router's operators and of AdamW: test infrastructure,
written from the formulas and independent of the HIP path.

Every function returns the values and, where a value is rounded on the GPU, a bound on the
error that fp32 arithmetic may make, in the comment's terms."""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
U = 2.0 ** -24  # half a step of fp32, relative


def clean(logits, mask=None):
    """f64 logits: NaN and masked rows -inf, +inf the largest finite f32."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, FLT_MAX))
    if mask is not None:
        x[np.asarray(mask) == 0] = -np.inf
    return x


def softmax(x):
    """(p, rel): row softmax (zeros for rows without a finite logit) and the relative error of
    an fp32 evaluation of each p. exp(d) of d = x - max: d is rounded by |d| U, which exp makes a
    relative error of |d| U; exp itself, the sum of up to 1024 terms over a tree and the quotient
    add under 40 U; the sum's own d errors average over p."""
    top = x.max(1)
    live = top > -np.inf
    d = x - np.where(live, top, 0.0)[:, None]
    e = np.exp(d)
    Z = np.where(live, e.sum(1), 1.0)[:, None]
    p = e / Z
    ad = np.where(np.isfinite(d), np.minimum(np.abs(d), 110.0), 0.0)  # beyond that p is 0 in fp32
    return p, (ad + (p * ad).sum(1, keepdims=True) + 40.0) * U


def route(logits, K, mask=None, first=0, local=None, renorm=False, scale=1.0):
    x = clean(logits, mask)
    T, E = x.shape
    local = E - first if local is None else local
    idx = np.full((T, K), -1, np.int32)
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:K]
        idx[t, :len(order)] = order
    ok = idx >= 0
    at = np.maximum(idx, 0)
    if renorm:
        p, rel = softmax(np.where(ok, np.take_along_axis(x, at, 1), -np.inf))
    else:
        pa, ra = softmax(x)
        p, rel = np.where(ok, np.take_along_axis(pa, at, 1), 0), np.take_along_axis(ra, at, 1)
    w = scale * p
    counts = np.bincount(idx[ok], minlength=E).astype(np.int32)
    seg, tok, slot, alpha = [0], [], [], []
    pmap = np.full((T, K), -1, np.int32)
    for e in range(first, first + local):
        for t, k in zip(*np.nonzero(idx == e)):
            pmap[t, k] = len(tok)
            tok.append(t)
            slot.append(k)
            alpha.append(w[t, k])
        seg.append(len(tok))
    return {"idx": idx, "w": w, "w_err": np.abs(w) * rel + 1e-37, "counts": counts, "seg_off": np.array(seg),
            "tok": np.array(tok, np.int32), "slot": np.array(slot, np.int32), "alpha": np.array(alpha), "pmap": pmap}


def balance(logits, idx, coef, mask=None, seq_off=None):
    x = clean(logits, mask)
    T, E = x.shape
    K = idx.shape[1]
    off = [0, T] if seq_off is None else list(seq_off)
    S = len(off) - 1
    p, rel = softmax(x) if T else (x, x)
    live = x.max(1) > -np.inf if T else np.zeros(0, bool)
    counts, psum, err, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros((S, E)), np.zeros(S)
    for s in range(S):
        rows = slice(off[s], off[s + 1])
        chosen = idx[rows][live[rows]]
        chosen = chosen[(chosen >= 0) & (chosen < E)]
        counts[s] = np.bincount(chosen.reshape(-1), minlength=E)
        psum[s], n[s] = p[rows].sum(0), live[rows].sum()
        # each p, sums of up to 256 of them in fp32, joins in fp64, one rounding
        err[s] = (p[rows] * (rel[rows] + 257 * U)).sum(0) + 1e-37
    alive = max(1, int((n > 0).sum()))
    norm = np.array([coef * E / (alive * K * v * v) if v else 0.0 for v in n])
    loss = float((norm[:, None] * counts * psum).sum())
    loss_err = float((np.abs(norm)[:, None] * counts * err).sum()) + 8 * U * abs(loss)
    return {"counts": counts, "psum": psum, "psum_err": err, "norm": norm, "loss": loss, "loss_err": loss_err}


def route_bwd(logits, idx, y=None, counts=None, norm=None, gloss=1.0, mask=None, seq_off=None, renorm=False,
              scale=1.0):
    """y [T, K]: the routing weights' gradient by slot. Returns (dlogits, err)."""
    x = clean(logits, mask)
    T, E = x.shape
    live = x.max(1) > -np.inf
    p, rel = softmax(x)
    dx, err = np.zeros((T, E)), np.zeros((T, E))
    if y is not None:
        d, chosen = np.zeros((T, E)), np.zeros((T, E), bool)
        for t in range(T):
            for k, e in enumerate(idx[t]):
                if 0 <= e < E and x[t, e] > -np.inf:
                    d[t, e], chosen[t, e] = scale * y[t, k], True
        q, qr = (softmax(np.where(chosen, x, -np.inf)) if renorm else (p, rel))
        s = (q * d).sum(1, keepdims=True)
        dx = q * (d - s)
        # relative errors of q twice (outside and in s), of the product with scale, and of the sum
        qr = qr + 48 * U
        err = q * (np.abs(d) * qr + (q * np.abs(d) * qr).sum(1, keepdims=True) + (q * np.abs(d)).sum(1, keepdims=True) * qr)
    if norm is not None:
        off = [0, T] if seq_off is None else list(seq_off)
        for s in range(len(off) - 1):
            r = slice(off[s], off[s + 1])
            c = counts[s].astype(np.float64)
            dot = (p[r] * c).sum(1, keepdims=True)
            f = norm[s] * gloss
            pr = rel[r] + 48 * U
            dx[r] += f * p[r] * (c - dot)
            err[r] += abs(f) * p[r] * (c * pr + (p[r] * c * pr).sum(1, keepdims=True) + dot * pr)
    dx[~live] = 0
    err += np.abs(dx) * U + 1e-37
    return dx, err


def alpha_grad(G, Y, alpha, tok, keep=None):
    """(dalpha, err): fp64 sums on the GPU too, so one rounding to f32 and fp64's own."""
    g, y = np.asarray(G, np.float64)[tok], np.asarray(Y, np.float64)
    a = np.asarray(alpha, np.float64)
    on = (a != 0) & (np.ones(len(a), bool) if keep is None else np.asarray(keep) != 0)
    safe = np.where(a != 0, a, 1.0)
    d = np.where(on, (g * y).sum(1) / safe, 0.0)
    mag = np.where(on, np.abs(g * y).sum(1) / np.abs(safe), 0.0)
    return d, np.abs(d) * U + mag * 2.0 ** -45


# ------------------------------------------------------------------------------- AdamW

BLOCK = 256


def adamw(w, g, m, v, *, lr, betas, eps, weight_decay, t, grad_scale=1.0):
    """fp64 step from the given state: (w, m, v) and bounds of fp32 arithmetic with a rounding at
    each operation and constants rounded to fp32."""
    b1, b2 = betas
    w, g, m, v = (np.asarray(a, np.float64) for a in (w, g, m, v))
    g = g * grad_scale
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    em = U * (2 * np.abs(b1 * m) + 4 * np.abs((1 - b1) * g) + np.abs(m1)) + 1e-44
    ev = U * (2 * b2 * v + 7 * (1 - b2) * g * g + v1) + 1e-44
    c1, c2 = 1 / (1 - b1 ** t), 1 / np.sqrt(1 - b2 ** t)
    r = np.sqrt(v1)
    den = r * c2 + eps
    u = np.divide(m1 * c1, den, out=np.zeros_like(m1), where=den > 0)
    w1 = w * (1 - lr * weight_decay) - lr * u
    er = np.divide(ev, 2 * r, out=np.zeros_like(r), where=r > 0) + U * r  # of the root
    eu = np.divide(em * c1, den, out=np.zeros_like(m1), where=den > 0) + np.abs(u) * (
        np.divide(er * c2, den, out=np.zeros_like(r), where=den > 0) + 8 * U)
    ew = lr * eu + U * (2 * np.abs(w) + 3 * np.abs(lr * u) + np.abs(w1)) + 1e-44
    return (w1, m1, v1), (ew, em, ev)


def mix(x):
    x = np.asarray(x, np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x85EBCA77)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(13))


def random_bits(n, first, seed, t):
    """(low, high) 16 bits of every element's word."""
    key = mix((int(seed) + int(mix(t & 0xFFFFFFFF))) & 0xFFFFFFFF)
    c = np.arange(n, dtype=np.uint64) + np.uint64(first)
    k = mix((key + (c >> np.uint64(32)) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF))
    h = mix(((c & np.uint64(0xFFFFFFFF)) + k) & np.uint64(0xFFFFFFFF))
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def quantise(x, bits, signed):
    """(values, scales): f32 x rounded at random to e4m3 values times a power of two per block."""
    x = np.asarray(x, np.float32)
    n = len(x)
    pad = -n % BLOCK
    a = np.concatenate([np.where(np.isfinite(x), np.abs(x), 0), np.zeros(pad)]).astype(np.float32).reshape(-1, BLOCK)
    amax = a.max(1)
    k = np.maximum(np.frexp((amax * np.float32(0.8164966)).astype(np.float64))[1] - 8, -126)
    scale = np.where(amax > 0, np.exp2(k.astype(np.float64)), 1.0)
    y = np.abs(x.astype(np.float64)) / np.repeat(scale, BLOCK)[:n]
    fin = np.isfinite(x)
    y = np.where(fin, y, 0)
    e = np.maximum(np.frexp(np.where(y > 0, y, 1.0))[1] - 1, -6)
    step = np.exp2(e - 3.0)
    # the sum is rounded to f32 like the kernel's
    q = np.floor((y / step).astype(np.float32) + ((bits + 0.5) / 65536).astype(np.float32)) * step
    if not signed:
        q = np.where(x > 0, np.maximum(q, 2.0 ** -9), q)
    return np.where(fin, np.where(signed & (x < 0), -q, q), np.nan), scale


def dequantise(q, scale):
    return np.asarray(q, np.float64) * np.repeat(np.asarray(scale, np.float64), BLOCK)[:len(q)]


def adamw_f32(g, m, v, betas, grad_scale=1.0):
    """The moments in f32 with a rounding at each operation, as the header fixes them: (m, v, r)."""
    f = np.float32
    b1, b2 = f(betas[0]), f(betas[1])
    a1, a2 = f(1 - betas[0]), f(1 - betas[1])
    g, m, v = (np.asarray(a, f) for a in (g, m, v))
    with np.errstate(over="ignore", invalid="ignore"):
        x = g * f(grad_scale)
        m1, v1 = m * b1 + x * a1, v * b2 + (x * x) * a2
        return m1, v1, np.sqrt(v1)
