"""Plain float64 definition of pa_logprobs (numpy), and the error that fp32
arithmetic may have in it."""
from __future__ import annotations

import numpy as np


def logprobs(logits, tokens, top, temperatures=None):
    """logits float64 values [rows, vocab].  Returns a dict: logprobs, entropy,
    top_ids, top_logprobs and the bounds tol_* on an fp32 evaluation.

    The bounds count roundings of 2^-24.  A weight 2^y, y = (x - max) log2(e)/T,
    has an error of the difference, of the factor (3 roundings with its own) and
    of ex2 (4): relative 2^-24 (4 |y| + 4).  A thread adds at most vocab/512
    pairs, then 20 partial sums are joined (3 roundings each).  So the sum is
    off by 2^-24 (vocab/512 + 64 + 4 sum p|y|) of it, the entropy's second sum,
    sum p y, by that times itself and by 2^-24 * 4 sum p y^2, and a log
    probability by the former plus the roundings of its own difference and
    quotient."""
    x = np.asarray(logits, np.float64)
    rows, vocab = x.shape
    t = np.ones(rows) if temperatures is None else np.asarray(temperatures, np.float64)
    u = 2.0 ** -24
    out = {k: np.zeros(rows) for k in ("logprobs", "entropy", "tol_logprobs", "tol_entropy")}
    out["top_ids"] = np.zeros((rows, top), np.int64)
    out["top_logprobs"], out["tol_top"] = np.zeros((rows, top)), np.zeros((rows, top))
    for r in range(rows):
        z, tok = x[r].copy(), int(tokens[r])
        z[z > -np.inf] /= t[r]  # -inf stays, under T = inf too
        # NaN last, then -inf; the sort is stable, so equal logits keep index order.
        order = np.argsort(-np.where(np.isnan(x[r]), -np.inf, x[r]), kind="stable")
        order = np.concatenate([order[~np.isnan(x[r][order])], order[np.isnan(x[r][order])]])[:top]
        if np.isnan(z).any() or (z == np.inf).any():
            lp, h, n, py, py2 = np.full(vocab, np.nan), np.nan, 0, 0, 0
            d = np.zeros(vocab)
        elif (z == -np.inf).all():
            lp, h, n, py, py2 = np.full(vocab, -np.inf), 0.0, 0, 0, 0
            d = np.zeros(vocab)
        else:
            d = z - z.max()
            w = np.exp(d)
            total = w.sum()
            p = w / total
            lp = d - np.log(total)
            fin = p > 0
            h = -(p[fin] * lp[fin]).sum()
            y = np.abs(d[fin]) / np.log(2.0)
            n, py, py2 = vocab / 512 + 64, (p[fin] * y).sum(), (p[fin] * y * y).sum()
        lp = np.where(lp < -np.finfo(np.float32).max, -np.inf, lp)  # what fp32 cannot hold
        out["logprobs"][r] = lp[tok] if 0 <= tok < vocab else -np.inf
        out["entropy"][r] = h
        out["top_ids"][r], out["top_logprobs"][r] = order, lp[order]
        base = u * (n + 4 * py + 4)
        dist = np.where(np.isfinite(d), np.abs(d), 0.0)
        tol = base + 4 * u * (dist + np.abs(np.where(np.isfinite(lp), lp, 0.0)))
        out["tol_logprobs"][r] = tol[tok] if 0 <= tok < vocab else 0.0
        out["tol_top"][r] = tol[order]
        out["tol_entropy"][r] = base * (2 + py) + 4 * u * (py2 + py + abs(h if np.isfinite(h) else 0.0))
    return out
