"""Beam search's selection over beams and vocabulary (oracle; test infrastructure only).

The rules of include/treeverify.h's tv_beam_select, one group at a time in plain Python, in fp64.
"""

import math

import numpy as np

OK, ERR_VALUE = 0, -11


def select_group(logits, scores, done, eos, scale):
    """logits [width, vocab], scores, done [width].  Returns (code, rows): per slot (source within the
    group, token, score, done, rank)."""
    width, code, found = len(scores), OK, []
    for w in range(width):
        if not scores[w] < math.inf:
            code = ERR_VALUE
            continue
        if scores[w] == -math.inf:
            continue
        if done[w]:
            found.append((-float(scores[w]), w, eos, 1))
            continue
        x = np.asarray(logits[w], dtype=np.float64)
        if np.isnan(x).any() or (x == math.inf).any():
            code = ERR_VALUE
            continue
        top = x.max()
        if top == -math.inf:
            continue
        lse = math.log(np.exp(scale * (x - top)).sum())
        order = np.lexsort((np.arange(len(x)), -x))[:width]
        found += [(-(float(scores[w]) + (scale * (x[t] - top) - lse)), w, int(t), int(t == eos))
                  for t in order if x[t] > -math.inf]
    found = sorted(found)[:width]
    slot_of, later = {}, []
    for k, f in enumerate(found):
        if f[1] in slot_of:
            later.append(k)
        else:
            slot_of[f[1]] = k
    empty = [w for w in range(width) if w not in slot_of]
    slot_of.update(zip(empty, later))
    rows = []
    for w in range(width):
        if w not in slot_of:
            rows.append((-1, -1, -math.inf, 0, -1))
        else:
            score, source, token, ended = found[slot_of[w]]
            rows.append((source, token, -score, ended, slot_of[w]))
    return code, rows
