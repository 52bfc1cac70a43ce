"""New tokens behind a committed prefix: their rows, the entries they complete, and what they attend to
(oracle; test infrastructure only).

The rules of include/treeverify.h's tv_chunk_append and tv_chunk_attn, request by request: the last
``rope_dim`` elements of a key (and of its token's queries) are rotated by position times inv_freq, the
rows and the entries of the blocks they complete are stored rounded to the cache's type, and a token
at position p sees the C4 entries below p // 4, the C128 entries below p // 128 and the raw rows
raw_lo(p) .. p ([TSD-V4] §2.2, §3.1: ordinary causal decoding).
"""

import math

import numpy as np

from .compress import gated_block_sum
from .storage import round_to_storage, to_f64


def rotate(rows, positions, rope_dim, pairs, inv_freq):
    """rows [n, ..., d] with the last rope_dim elements of row i rotated by positions[i], unrounded."""
    out = to_f64(rows).copy()
    first = out.shape[-1] - rope_dim
    for i, p in enumerate(positions):
        for k in range(rope_dim // 2):
            a = float(p) * float(inv_freq[k])
            x, y = (first + 2 * k, first + 2 * k + 1) if pairs else (first + k, first + rope_dim // 2 + k)
            u, v = out[i, ..., x].copy(), out[i, ..., y].copy()
            out[i, ..., x] = u * math.cos(a) - v * math.sin(a)
            out[i, ..., y] = u * math.sin(a) + v * math.cos(a)
    return out


def append_request(rawK, rawV, comp, L, K, V, g, store, rope_dim=0, pairs=0, inv_freq=()):
    """rawK, rawV [cap, d] and comp {m: (CK, CV)} are changed in place; returns the new length."""
    n = len(K)
    rawK[L:L + n] = round_to_storage(rotate(K, range(L, L + n), rope_dim, pairs, inv_freq), store)
    rawV[L:L + n] = to_f64(V)
    for m, (CK, CV) in comp.items():
        for j in range(L // m, (L + n) // m):
            ck, cv = gated_block_sum(rawK[m * j:m * j + m], rawV[m * j:m * j + m], g[m])
            CK[j], CV[j] = round_to_storage(ck, store), round_to_storage(cv, store)
    return L + n


def seen(p, rawK, rawV, comp, W, tail_mode):
    """The rows a token at position p attends to: (K, V), fp64."""
    lo = max(0, p - W) if tail_mode == "window" else min(comp) * (p // min(comp))
    K = [to_f64(CK[:p // m]) for m, (CK, _) in sorted(comp.items())] + [to_f64(rawK[lo:p + 1])]
    V = [to_f64(CV[:p // m]) for m, (_, CV) in sorted(comp.items())] + [to_f64(rawV[lo:p + 1])]
    return np.concatenate(K), np.concatenate(V)


def attend_request(Q, L, rawK, rawV, comp, W, tail_mode, scale):
    """Q [n, H, d] belongs to the last n of L positions.  Returns O [n, H, d], lse [n, H] and, for the
    tests' tolerances, sum_j p_j |v_j| and the largest sum_i |q_i k_i| * scale of every row."""
    n, H, d = Q.shape
    O, lse = np.zeros((n, H, d)), np.zeros((n, H))
    spread, size = np.zeros((n, H, d)), np.zeros((n, H))
    for i in range(n):
        K, V = seen(L - n + i, rawK, rawV, comp, W, tail_mode)
        q = to_f64(Q[i])
        s = (q @ K.T) * scale
        m = s.max(axis=1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(axis=1, keepdims=True)
        O[i], lse[i] = (e @ V) / z, (m + np.log(z))[:, 0]
        spread[i] = (e @ np.abs(V)) / z
        size[i] = (np.abs(q) @ np.abs(K).T).max(axis=1) * scale
    return O, lse, spread, size
