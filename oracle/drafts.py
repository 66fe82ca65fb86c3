"""Speculative decoding over the pool, in float64: rotation, trees, attention of
drafted tokens, verification, compaction.  Written from the definitions; shares
no code with the kernels."""
import math

import numpy as np


# --------------------------------------------------------------------------
# Rotation
# --------------------------------------------------------------------------

def frequencies(rotary, theta, scaling=None):
    """(f_i in radians per position, gain)."""
    f, gain = [], 1.0
    kind = scaling[0] if scaling else None
    for i in range(rotary // 2):
        if kind == "ntk":
            f.append((theta * scaling[1] ** (rotary / (rotary - 2))) ** (-2 * i / rotary))
            continue
        x = theta ** (-2 * i / rotary)
        if kind == "linear":
            x = x / scaling[1]
        elif kind == "yarn":
            fast, slow = scaling[3:] if len(scaling) > 3 else (32.0, 1.0)
            dim = lambda beta: rotary * math.log(scaling[2] / (2 * math.pi * beta)) / (2 * math.log(theta))
            lo, hi = max(0, math.floor(dim(fast))), min(rotary - 1, math.ceil(dim(slow)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            x = x * (1 - r) + x / scaling[1] * r
            gain = 0.1 * math.log(scaling[1]) + 1
        f.append(x)
    return np.array(f), gain


def rope(x, positions, rotary, theta, scaling=None, interleaved=False, weight=None, eps=1e-6):
    """x [N, heads, 128] rotated, and a bound of an fp32 evaluation rounded once
    to bf16.

    Per value, in units of 2^-24: the sum of squares 19 roundings and eps 1,
    halved by the root, the root itself 4, two products: 16 relative in x.  The
    angle: one rounding of at most half a turn, pi; sincospi 4; the gain 1; the
    products and their sum 3.  28 < 2^-19 of g (|x1| + |x2|), then half a bf16
    step, 2^-8, of the result."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    f, gain = frequencies(rotary, theta, scaling)
    angle = np.asarray(positions, np.float64)[:, None, None] * f
    c, s = np.cos(angle), np.sin(angle)
    first = slice(0, rotary, 2) if interleaved else slice(0, rotary // 2)
    second = slice(1, rotary, 2) if interleaved else slice(rotary // 2, rotary)
    y, size = x.copy(), np.abs(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = gain * (a * c - b * s), gain * (b * c + a * s)
    size[..., first] = size[..., second] = gain * (np.abs(a) + np.abs(b))
    t = 2.0 ** -19 * size
    if weight is None:
        t[..., rotary:] = 0  # copied
    return y, t + 2.0 ** -8 * (np.abs(y) + t) + 2.0 ** -133


# --------------------------------------------------------------------------
# Trees
# --------------------------------------------------------------------------

def random_parents(rng, n, reach=4):
    """A tree of n nodes, each under one of the `reach` nodes before it."""
    return np.array([-1] + [rng.integers(max(0, i - reach), i) for i in range(1, n)], np.int32)


def ancestors(parents):
    """sees[i, j]: j is i or an ancestor of i; and the depths."""
    n = len(parents)
    sees, depth = np.zeros((n, n), bool), np.zeros(n, np.int32)
    for i in range(n):
        if i:
            sees[i] = sees[parents[i]]
            depth[i] = depth[parents[i]] + 1
        sees[i, i] = True
    return sees, depth


def as_bits(sees):
    """int64 masks of boolean rows [n, <= 64]."""
    out = np.zeros(len(sees), np.uint64)
    for j in range(sees.shape[1]):
        out |= sees[:, j].astype(np.uint64) << np.uint64(j)
    return out.view(np.int64)


def attend(q, k, v, sees, scale):
    """One kv head of one sequence: q [n, G, 128], k and v [ctx, 128], sees [n, n]
    over the last n keys.  Outputs [n, G, 128] and a bound for an evaluation with
    fp32 scores and bf16 weights.

    A weight is off by half a bf16 step, 2^-8, and by its score's error: the
    product's 2^-19 of sum |q k| (eight steps of 16, each off by a few 2^-24 of
    its largest sum), 2^-22 of the score (its scaling) and 2^-20 (the power of two, as
    often as a maximum moves or parts meet).  With weights off by delta, each, and
    their sum with them, an output is off by delta * sum w |v - out|; sums of
    products in fp32 add 2^-18 sum w |v|, and the result's rounding 2^-8 of it."""
    n, G, _ = q.shape
    ctx = len(k)
    see = np.ones((n, ctx), bool)
    see[:, ctx - n:] = sees
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        at = np.nonzero(see[i])[0]
        if len(at) == 0:
            continue
        kk, vv = k[at], v[at]
        with np.errstate(invalid="ignore", over="ignore"):
            s = q[i] @ kk.T * scale
            size = np.abs(q[i]) @ np.abs(kk).T * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            w = w / w.sum(-1, keepdims=True)
            o = w @ vv
            delta = 2.0 ** -8 + 2 * (2.0 ** -19 * size + 2.0 ** -22 * np.abs(s) + 2.0 ** -20)
            spread = np.stack([(w[g] * delta[g]) @ np.abs(vv - o[g]) for g in range(G)])
            t = 1.02 * spread + 2.0 ** -18 * (w @ np.abs(vv)) + 2.0 ** -100
        out[i], tol[i] = o, t + 2.0 ** -8 * (np.abs(o) + t)
    return out, tol


def rows_of(cache, table, n):
    """Rows of positions 0..n-1: cache [num_blocks, B, Hkv, 128] -> [n, Hkv, 128]."""
    B = cache.shape[1]
    p = np.arange(n)
    return cache[table[p // B], p % B]


def decode_tree(q, kc, vc, tables, ctx, sees, scale, lens=None):
    """q [batch, T, Hq, 128]; sees: a list of boolean [n_b, n_b]."""
    batch, T, hq, _ = q.shape
    hkv = kc.shape[2]
    G = hq // hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(batch):
        n = (T if ctx[b] else 0) if lens is None else int(lens[b])
        if n == 0:
            continue
        k, v = rows_of(kc, tables[b], ctx[b]), rows_of(vc, tables[b], ctx[b])
        for h in range(hkv):
            hs = slice(h * G, (h + 1) * G)
            out[b, :n, hs], tol[b, :n, hs] = attend(q[b, :n, hs], k[:, h], v[:, h], sees[b][:n, :n], scale)
    return out, tol


# --------------------------------------------------------------------------
# Verification
# --------------------------------------------------------------------------

def verify(logits, tokens, parents, u, noise, temps, probs=None, lens=None):
    """Returns tokens, nodes, counts and, per sequence, the smallest relative
    distance of any of its decisions from the other way."""
    batch, T, vocab = logits.shape
    out_t, out_n = np.full((batch, T), -1, np.int32), np.full((batch, T), -1, np.int32)
    counts, margin = np.zeros(batch, np.int32), np.full(batch, np.inf)
    for b in range(batch):
        n = T if lens is None else int(lens[b])
        if n == 0:
            continue
        path, v, kept = [0], 0, []
        while True:
            z = np.asarray(logits[b, v], np.float64)
            z = np.where(np.isnan(z), -np.inf, np.minimum(z, float(np.finfo(np.float32).max))) / float(temps[b])
            top = z.max()
            p = np.zeros(vocab) if top == -np.inf else np.exp(z - top) / np.exp(z - top).sum()
            w, nxt = p, None
            for c in range(v + 1, n):
                if parents[b][c] != v:
                    continue
                x = tokens[b][c]
                if not 0 <= x < vocab:
                    continue
                q = np.zeros(vocab)
                if probs is None:
                    q[x] = 1.0
                else:
                    q = np.asarray(probs[b, v], np.float64)
                total = 1.0 if w is p else w.sum()
                a, d = float(u[b][c]) * q[x] * total, w[x]
                if max(a, d) > 0:
                    margin[b] = min(margin[b], abs(a - d) / max(a, d))
                if a < d:
                    nxt = c
                    break
                if probs is None:
                    w = np.where(np.arange(vocab) == x, 0.0, w)
                else:
                    w = np.maximum(w - total * q, 0.0)
            if nxt is None:
                break
            kept.append(tokens[b][nxt])
            path.append(nxt)
            v = nxt
        if not np.any(w > 0):
            w = p
        r = w / np.maximum(np.asarray(noise[b], np.float64), 1e-10)
        best = int(np.argmax(r))
        if r[best] > 0 and vocab > 1:
            margin[b] = min(margin[b], 1 - np.partition(r, -2)[-2] / r[best])
        counts[b] = len(path)
        out_n[b, :len(path)] = path
        out_t[b, :len(path)] = kept + [best]
    return out_t, out_n, counts, margin


# --------------------------------------------------------------------------
# Compaction
# --------------------------------------------------------------------------

def compact(cache, tables, ctx, nodes, counts, lens=None):
    """cache [num_blocks, B, ...] with the kept rows moved; a new array."""
    out = cache.copy()
    B = cache.shape[1]
    for b in range(len(ctx)):
        n = (nodes.shape[1] if ctx[b] else 0) if lens is None else int(lens[b])
        base = int(ctx[b]) - n
        for j in range(min(int(counts[b]), n)):
            s, d = base + int(nodes[b, j]), base + j
            out[tables[b][d // B], d % B] = cache[tables[b][s // B], s % B]
    return out
