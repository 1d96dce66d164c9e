"""Sampling one token per row, written plainly in binary64.

TEST INFRASTRUCTURE ONLY: the reference the library's sampling kernels are checked against.

w_v = exp((z_v - max z) / T); tokens rank by logit, equal logits by the smaller id; top-k keeps the
first k ranks, top-p the shortest run of leading ranks with p / 1000 of the top-k mass, min-p the
tokens with w >= min_p; the token is min{v : C(v) > u S} in ascending id over the kept weights.
"""
from __future__ import annotations

import numpy as np


def sample_row(z, u, T, top_k=0, top_p_milli=1000, min_p=0.0) -> dict:
    """token, probs [V], kept count, and margin: the distance of u to the nearest border of the
    distribution function (the draw is certain beyond the rounding of the sums)."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64))
    V = z.shape[0]
    nothing = {"token": -1, "probs": np.zeros(V), "kept": 0, "margin": 1.0, "prob": 0.0}
    if not (T >= 0 and np.isfinite(T)) or not np.isfinite(z.max()):
        return nothing
    if T == 0:
        probs = np.zeros(V)
        probs[int(z.argmax())] = 1.0
        return {"token": int(z.argmax()), "probs": probs, "kept": 1, "margin": 1.0, "prob": 1.0}
    if top_k < 0 or not 0 <= top_p_milli <= 1000 or not 0 <= min_p <= 1 or not 0 <= u < 1:
        return nothing
    with np.errstate(over="ignore"):
        w = np.exp((z - z.max()) / np.float64(T))
    order = np.lexsort((np.arange(V), -z))
    keep = top_k if 0 < top_k < V else V
    if top_p_milli < 1000:
        run = np.cumsum(w[order[:keep]])
        keep = min(keep, int(np.sum(run * 1000 < top_p_milli * run[-1])) + 1)
    if min_p > 0:
        keep = min(keep, int(np.sum(w >= np.float64(np.float32(min_p)))))
    kept = np.zeros(V, dtype=bool)
    kept[order[:keep]] = True
    w = np.where(kept, w, 0.0)
    c = np.cumsum(w)
    y = int(np.sum(c <= u * c[-1]))
    y = min(y, int(np.flatnonzero(w > 0)[-1]))
    return {"token": y, "probs": w / c[-1], "kept": keep, "margin": float(np.min(np.abs(c / c[-1] - u))),
            "prob": w[y] / c[-1]}
