"""From logits to targets, alternatives and log probabilities (oracle; test infrastructure only).

Greedy verification needs the largest logit of every tree node ([TSD-V4] §3.2); growing a draft
tree needs the best alternatives with their probabilities, and judging one the log probabilities
of its tokens.  Everything is the plain definition over softmax(scale * x), one row at a time, in
fp64; the logits are the stored values, so the integer outputs are decided without rounding.
"""

import math

import numpy as np


def row_logprobs(x, scale):
    """(lse, entropy, logp [V]) of one row of logits."""
    z = np.asarray(x, dtype=np.float64) * scale
    if np.isnan(z).any() or np.isposinf(z).any():
        return math.nan, math.nan, np.full(z.shape, math.nan)
    m = z.max()
    if m == -math.inf:
        return -math.inf, 0.0, np.full(z.shape, -math.inf)
    log_s = math.log(np.exp(z - m).sum())
    logp = (z - m) - log_s
    p = np.exp(logp)
    seen = p > 0
    return m + log_s, float(-(p[seen] * logp[seen]).sum()), logp


def row_order(x):
    """Ids of the logits above -inf, largest first, equal logits by id (empty with a NaN or +inf)."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.zeros(0, dtype=np.int64)
    ids = np.flatnonzero(x > -math.inf)
    return ids[np.lexsort((ids, -x[ids]))]


def token_logprobs(logits, tokens=None, nodes=None, scale=1.0, n_top=0):
    """logits [B, D, V]; tokens, nodes [B, n] (nodes None: entry i is on node i; negative: 0).
    Returns lse, entropy [B, D], target [B, D], top_ids, top_logprobs [B, D, n_top], logprobs
    [B, n] as fp64 / int64 arrays."""
    B, D, _ = logits.shape
    n = 0 if tokens is None else tokens.shape[1]
    out = dict(lse=np.zeros((B, D)), entropy=np.zeros((B, D)),
               target=np.full((B, D), -1, dtype=np.int64),
               top_ids=np.full((B, D, n_top), -1, dtype=np.int64),
               top_logprobs=np.full((B, D, n_top), -math.inf), logprobs=np.zeros((B, n)))
    for b in range(B):
        for v in range(D):
            x = np.asarray(logits[b, v], dtype=np.float64)
            lse, h, logp = row_logprobs(x, scale)
            ids = row_order(x)
            out["lse"][b, v], out["entropy"][b, v] = lse, h
            if len(ids):
                out["target"][b, v] = ids[0]
            k = min(n_top, len(ids))
            out["top_ids"][b, v, :k] = ids[:k]
            out["top_logprobs"][b, v, :k] = logp[ids[:k]]
            if math.isnan(lse):
                out["top_logprobs"][b, v] = math.nan
            for i in range(n):
                node = i if nodes is None else int(nodes[b, i])
                if node == v and tokens[b, i] >= 0:
                    out["logprobs"][b, i] = logp[int(tokens[b, i])]
    return out
