"""Float64 CPU oracle for drawing tokens under temperature, top-k, top-p and
min-p (test infrastructure, not product code; shares nothing with the CUDA
library)."""
from __future__ import annotations

import math

import numpy as np

SUPPORT = 2.0 ** -40


def ref_sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probs, gap, weight) of one row.  weight is the total kept
    weight in units of the largest; gap is the distance of the nearest
    border that decided the result, as a share of the total weight: the steps of
    the distribution on both sides of u, and for top-p the weight by which the
    border token passes (or the one before it misses) the asked share."""
    x = np.asarray(logits, dtype=np.float64)
    V = len(x)
    valid = ~np.isnan(x)
    m = np.max(x[valid]) if valid.any() else -math.inf
    tau = float(np.float32(temperature))
    if not math.isfinite(m) or math.isnan(tau) or tau == math.inf:
        return -1, np.zeros(V), 1.0, 1.0
    if tau < 2.0 ** -64:
        v = int(np.flatnonzero(x == m)[0])
        return v, (np.arange(V) == v).astype(np.float64), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(valid, np.exp((x - m) / tau), 0.0)
        order = np.sort(np.where(valid, x, -math.inf))[::-1]
        kept = valid & (w >= SUPPORT)
        if 0 < top_k < V:
            in_k = valid & (x >= order[top_k - 1])
        else:
            in_k = valid.copy()
    in_k &= w >= SUPPORT
    kept &= in_k
    gap = 1.0
    p = float(np.float32(top_p))
    if p < 1:
        xs = np.sort(x[in_k])[::-1]
        cum = np.cumsum(np.exp((xs - m) / tau))
        # the last of equal logits stands for them all
        last = np.append(xs[1:] != xs[:-1], True)
        xs, cum = xs[last], cum[last]
        at = min(int(np.searchsorted(cum, p * cum[-1])), len(xs) - 1) if p > 0 else 0
        kept &= x >= xs[at]
        if p > 0:
            gap = min(gap, abs(cum[at] - p * cum[-1]) / cum[-1])
            if at:
                gap = min(gap, abs(cum[at - 1] - p * cum[-1]) / cum[-1])
    low = float(np.float32(min_p))
    if low > 0:
        floor = min(low, 1.0)
        kept &= w >= floor
        near = np.abs(w - floor) / floor
        near[w == floor] = 1.0
        gap = min(gap, float(near.min()))
    ids = np.flatnonzero(kept)
    cum = np.cumsum(w[ids])
    u = 0.0 if not float(u) > 0 else min(float(u), 1.0)
    at = min(int(np.searchsorted(cum, u * cum[-1], side="right")), len(ids) - 1)
    gap = min(gap, abs(cum[at] - u * cum[-1]) / cum[-1])
    if at:
        gap = min(gap, abs(cum[at - 1] - u * cum[-1]) / cum[-1])
    probs = np.zeros(V)
    probs[ids] = w[ids] / cum[-1]
    return int(ids[at]), probs, gap, cum[-1]


def ref_sample_tokens(logits, uniforms, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Rows of ref_sample_row: (tokens [T], probs [T, V], gaps [T], weights [T]); every
    setting a number or one per row."""
    T = len(logits)
    rows = [np.broadcast_to(np.asarray(s), (T,)) for s in (temperature, top_k, top_p, min_p)]
    out = [ref_sample_row(logits[t], uniforms[t], rows[0][t], int(rows[1][t]), rows[2][t], rows[3][t]) for t in range(T)]
    return np.array([o[0] for o in out]), np.stack([o[1] for o in out]), np.array([o[2] for o in out]), np.array([o[3] for o in out])
