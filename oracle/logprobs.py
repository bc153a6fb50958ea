"""Oracle: log probabilities of given tokens, entropy and top alternatives
(test infrastructure).

"Encode branch histories in masks and positions": node i's logits predict the
token emitted at it, so the entry (token, node) of an accepted path has log
probability ``log_softmax(logits[node])[token]``.  Entropy is
``-sum p ln p`` with ``0 ln 0 = 0``; alternatives are the largest logits,
equal ones by ascending index.  A logit of -inf has probability 0.  A row
without a distribution (all -inf, or a NaN or +inf in it) has NaN everywhere
but in its alternatives' order, where a NaN ranks as -inf.  An entry whose
token or node is negative or out of range is no entry: 0, 0, -1 and -inf.
"""

from __future__ import annotations

import numpy as np


def token_logprobs(logits, tokens, node=None, top_k=0):
    """logits [B, N, V], tokens [B, C], node [B, C] (None: column c reads row c)
    -> (logprob [B, C], entropy [B, C], top_ids [B, C, K], top_logprobs [B, C, K]), float64."""
    B, N, V = logits.shape
    C = tokens.shape[1]
    lp, ent = np.zeros((B, C)), np.zeros((B, C))
    ids = np.full((B, C, top_k), -1, dtype=np.int32)
    top = np.full((B, C, top_k), -np.inf)
    for b in range(B):
        for c in range(C):
            r, tok = (c if node is None else int(node[b, c])), int(tokens[b, c])
            if not (0 <= r < N and 0 <= tok < V):
                continue
            x = np.asarray(logits[b, r], dtype=np.float64)
            rank = np.where(np.isnan(x), -np.inf, x)
            order = np.lexsort((np.arange(V), -rank))[:top_k]
            ids[b, c] = order
            if np.isnan(x).any() or not np.isfinite(x.max()):
                lp[b, c] = ent[b, c] = np.nan
                top[b, c] = np.nan
                continue
            e = np.exp(x - x.max())
            logp = x - x.max() - np.log(e.sum())
            p = e / e.sum()
            lp[b, c] = logp[tok]
            ent[b, c] = -(p[p > 0] * logp[p > 0]).sum()
            top[b, c] = logp[order]
    return lp, ent, ids, top
