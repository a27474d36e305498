"""Plain fp64 numpy definitions of routing by scores (softmax or sigmoid, bias, groups), of the balance loss of
sigmoid scores, of both gradients and of the bias update: test infrastructure, written from the formulas and
independent of the HIP path. Values that are rounded on the GPU come with a bound on the error of fp32 arithmetic."""
from __future__ import annotations

import numpy as np

from .router_oracle import FLT_MAX, U, clean, softmax


def sigmoid(x):
    x = np.asarray(x, np.float64)
    z = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, z) / (1.0 + z)


def shares(x, score):
    """(p, rel): scores of a row over their sum (zeros for rows without a logit over -inf), and the relative error of an
    fp32 evaluation. Sigmoid: each term is exp(d) / (1 + exp(-|x|)) with d = min(x, 0) - min(max, 0), whose rounding is a
    relative |d| U; the exponentials (2 ulp each, and |x| exp(-|x|) < 0.4 of the second's argument), sum, reciprocal and
    product of a term stay under 14 U, the sum over a tree and the quotient add under 12 U, and the sum's errors average
    over p: 40 U in all beside the d terms. Terms below 2^-126 of the largest count as 0: 2^-126 absolute."""
    if score == "softmax":
        return softmax(x)
    top = x.max(1)
    live = top > -np.inf
    low = np.minimum(x, 0)
    d = low - np.where(live, np.minimum(top, 0), 0)[:, None]
    e = np.where(x > -np.inf, np.exp(d) / (1 + np.exp(-np.abs(x))), 0.0)
    p = e / np.where(live, e.sum(1), 1.0)[:, None]
    ad = np.where(np.isfinite(d), np.minimum(np.abs(d), 110.0), 0.0)
    return p, (ad + (p * ad).sum(1, keepdims=True) + 40.0) * U


def choice_scores(x, score, bias=None):
    """f64 choice scores of clean logits, -inf for what is no candidate."""
    s = sigmoid(x) if score == "sigmoid" else softmax(x)[0]
    b = np.zeros(x.shape[1]) if bias is None else clean(np.asarray(bias, np.float64)[None])[0]
    return np.where((x > -np.inf) & (b > -np.inf)[None], s + np.where(b > -np.inf, b, 0)[None], -np.inf)


# The GPU compares choice scores to 42 bits and group sums to 44, so those that agree to this, relative, may come in
# either order.
NEAR = 2.0 ** -41


def _of_groups(c, groups, group_best):
    size, found = len(c) // groups, []
    for g in range(groups):
        best = sorted((v for v in c[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:group_best]
        found.append(sum(best) if best else -np.inf)
    return found


def _check_near(c, scores, by_logit, idx, groups, top_groups, group_best):
    """That the choice of a token is one of those that NEAR allows; logits are compared exactly."""
    size, chosen = len(c) // groups, [int(e) for e in idx if e >= 0]
    of_group = _of_groups(scores, groups, group_best)
    there = sorted((g for g in range(groups) if of_group[g] > -np.inf), key=lambda g: (-of_group[g], g))
    kept = there[:top_groups]
    if len(there) > top_groups:
        border = of_group[kept[-1]]
        near = [g for g in there if abs(of_group[g] - border) <= NEAR * abs(border)]
        used = sorted({e // size for e in chosen})
        sure = [g for g in kept if g not in near]
        assert set(used) <= set(sure) | set(near)
        kept = (sure + [g for g in near if g in used] + [g for g in near if g not in used])[:top_groups]
        assert set(used) <= set(kept)
    left = [e for g in kept for e in range(g * size, (g + 1) * size) if c[e] > -np.inf]
    assert len(set(chosen)) == len(chosen) == min(len(idx), len(left)) and set(chosen) <= set(left)
    for k, e in enumerate(chosen):
        best = max(c[f] for f in left if f not in chosen[:k])
        assert c[e] >= best - (0 if by_logit else NEAR * abs(best))


def route(logits, K, score, bias=None, groups=1, top_groups=1, group_best=1, mask=None, first=0, local=None, renorm=False,
          scale=1.0, given=None):
    """``given``: a choice [T, K] that is checked and taken where it differs within NEAR."""
    x = clean(logits, mask)
    T, E = x.shape
    local, size = E - first if local is None else local, E // groups
    scores = choice_scores(x, score, bias)
    c = x if bias is None else scores  # without a bias by the logits, whose order is that of the scores
    idx = np.full((T, K), -1, np.int32)
    for t in range(T):
        of_group = _of_groups(scores[t], groups, group_best)
        kept = sorted((g for g in range(groups) if of_group[g] > -np.inf), key=lambda g: (-of_group[g], g))[:top_groups]
        order = sorted((e for g in kept for e in range(g * size, (g + 1) * size) if c[t, e] > -np.inf),
                       key=lambda e: (-c[t, e], e))[:K]
        idx[t, :len(order)] = order
        if given is not None and not np.array_equal(given[t], idx[t]):
            _check_near(c[t], scores[t], bias is None, given[t], groups, top_groups, group_best)
            idx[t] = given[t]
    ok = idx >= 0
    at = np.maximum(idx, 0)
    xk = np.where(ok, np.take_along_axis(x, at, 1), -np.inf)
    if renorm:
        p, rel = shares(xk, score)
    elif score == "sigmoid":
        p, rel = np.where(ok, sigmoid(xk), 0), np.full(xk.shape, 40 * U)
    else:
        pa, ra = softmax(x)
        p, rel = np.where(ok, np.take_along_axis(pa, at, 1), 0), np.take_along_axis(ra, at, 1)
    w = scale * p
    seg, tok, slot, alpha = [0], [], [], []
    pmap = np.full((T, K), -1, np.int32)
    for e in range(first, first + local):
        for t, k in zip(*np.nonzero(idx == e)):
            pmap[t, k] = len(tok)
            tok.append(t)
            slot.append(k)
            alpha.append(w[t, k])
        seg.append(len(tok))
    return {"idx": idx, "w": w, "w_err": np.abs(w) * rel + 1e-37, "seg_off": np.array(seg),
            "counts": np.bincount(idx[ok], minlength=E).astype(np.int32), "tok": np.array(tok, np.int32),
            "slot": np.array(slot, np.int32), "alpha": np.array(alpha), "pmap": pmap}


def balance(logits, idx, coef, score, mask=None, seq_off=None):
    x = clean(logits, mask)
    T, E = x.shape
    K = idx.shape[1]
    off = [0, T] if seq_off is None else list(seq_off)
    S = len(off) - 1
    p, rel = shares(x, score)
    live = x.max(1) > -np.inf
    counts, psum, err, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros((S, E)), np.zeros(S)
    for s in range(S):
        r = slice(off[s], off[s + 1])
        chosen = idx[r][live[r]]
        counts[s] = np.bincount(chosen[(chosen >= 0) & (chosen < E)].reshape(-1), minlength=E)
        psum[s], n[s] = p[r].sum(0), live[r].sum()
        # each p, sums of up to 256 of them in fp32, joins in fp64, one rounding
        err[s] = (p[r] * (rel[r] + 257 * U)).sum(0) + 1e-37
    alive = max(1, int((n > 0).sum()))
    norm = np.array([coef * E / (alive * K * v * v) if v else 0.0 for v in n])
    loss = float((norm[:, None] * counts * psum).sum())
    loss_err = float((np.abs(norm)[:, None] * counts * err).sum()) + 8 * U * abs(loss)
    return {"counts": counts, "psum": psum, "psum_err": err, "norm": norm, "loss": loss, "loss_err": loss_err}


def sigmoid_bwd(logits, idx, y=None, counts=None, norm=None, gloss=1.0, mask=None, seq_off=None, renorm=False,
                scale=1.0):
    """y [T, K]: the routing weights' gradient by slot. Returns (dlogits, err). The factor 1 - s = sigmoid(-x) has a
    relative error under 12 U."""
    x = clean(logits, mask)
    T, E = x.shape
    live = x.max(1) > -np.inf
    away = np.where(x > -np.inf, sigmoid(-x), 0.0)
    dx, err = np.zeros((T, E)), np.zeros((T, E))
    if y is not None:
        d, chosen = np.zeros((T, E)), np.zeros((T, E), bool)
        for t in range(T):
            for k, e in enumerate(idx[t]):
                if 0 <= e < E and x[t, e] > -np.inf:
                    d[t, e], chosen[t, e] = scale * y[t, k], True
        if renorm:
            q, qr = shares(np.where(chosen, x, -np.inf), "sigmoid")
            s = (q * d).sum(1, keepdims=True)
            qr = qr + 60 * U
            mean = (q * np.abs(d)).sum(1, keepdims=True)
            err = q * away * (np.abs(d) * qr + (q * np.abs(d) * qr).sum(1, keepdims=True) + mean * qr)
        else:
            q, s = np.where(chosen, sigmoid(x), 0), 0.0
            err = q * away * np.abs(d) * 100 * U
        dx = np.where(chosen, q * away * (d - s), 0)
    if norm is not None:
        p, rel = shares(x, "sigmoid")
        off = [0, T] if seq_off is None else list(seq_off)
        for s in range(len(off) - 1):
            r = slice(off[s], off[s + 1])
            c = counts[s].astype(np.float64)
            dot = (p[r] * c).sum(1, keepdims=True)
            f = norm[s] * gloss
            pr = rel[r] + 60 * U
            dx[r] += f * p[r] * away[r] * (c - dot)
            err[r] += abs(f) * p[r] * away[r] * (c * pr + (p[r] * c * pr).sum(1, keepdims=True) + dot * pr)
    dx[~live] = 0
    err += np.abs(dx) * U + 1e-37
    return dx, err


def bias_update(bias, counts, rate):
    """f32 values: one rounding of the sum."""
    n = [int(v) for v in counts]
    step = np.array([(sum(n) > len(n) * v) * 1.0 - (sum(n) < len(n) * v) for v in n])
    return (np.asarray(bias, np.float32) + np.float32(rate) * step.astype(np.float32)).astype(np.float32)


__all__ = ["FLT_MAX", "U", "sigmoid", "shares", "choice_scores", "route", "balance", "sigmoid_bwd", "bias_update"]
