"""Oracle: a token drawn from a processed row of logits (test infrastructure).

"Implement the lossless speculative sampling verifier for a batch with ragged
draft lengths", *Details that matter in review*: acceptance compares the
distributions that tokens are really drawn from, so temperature, top-k, min-p
and top-p are applied first.  With w_i = e^((x_i - max x) / T): the top_k
largest logits stay (equal ones by index), of these the ones with w >= min_p,
of these in descending order the shortest run whose sum reaches top_p of
theirs; the token is the first index whose running sum over the kept w exceeds
u times their total.  T = 0 keeps the first largest logit.  A row with a NaN or
+inf, or nothing above -inf, or a temperature that is negative or not finite,
has no distribution: token -1, probabilities NaN.
"""

from __future__ import annotations

import math

import numpy as np


def processed(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Kept weights of one row [V] in float64 (None without a distribution)."""
    x = np.asarray(x, dtype=np.float64)
    V = x.size
    if np.isnan(x).any() or not np.isfinite(x.max()) or not (0.0 <= temperature < math.inf):
        return None
    order = np.lexsort((np.arange(V), -x))
    w = np.zeros(V)
    if temperature < 2.0 ** -60:
        w[order[0]] = 1.0
        return w
    e = np.exp((x[order] - x[order[0]]) / min(temperature, 2.0 ** 60))
    n = V if top_k <= 0 else min(top_k, V)
    e = e[:n]
    if min_p > 0.0:
        e = e[e >= min(min_p, 1.0)]
    if top_p < 1.0:
        before = np.concatenate(([0.0], np.cumsum(e)[:-1]))
        e = e[:max(1, int((before < top_p * e.sum()).sum()))]
    w[order[:e.size]] = e
    return w


def token_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """logits [R, V], u [R], the others [R] or None -> (tokens [R] int32, probs [R, V] float64)."""
    R, V = logits.shape
    tokens, probs = np.full(R, -1, dtype=np.int32), np.full((R, V), np.nan)
    for r in range(R):
        w = processed(logits[r], *(d if a is None else type(d)(a[r]) for a, d in
                                   ((temperature, 1.0), (top_k, 0), (top_p, 1.0), (min_p, 0.0))))
        if w is None:
            continue
        run = np.cumsum(w)
        goal = 0.0 if not u[r] > 0.0 else float(u[r]) * run[-1]
        hit = np.flatnonzero(run > goal)
        tokens[r] = hit[0] if hit.size and u[r] < 1.0 else np.flatnonzero(w)[-1 if u[r] >= 1.0 else 0]
        probs[r] = w / run[-1]
    return tokens, probs
