"""Pages of the pools: branching, reserving, compacting (oracle; test infrastructure only).

The report's cache is "one logical layer over three physical layers with shared page pointers"
([TSD-V4] §4.2); who owns which page is left to its serving engine.  These are the rules of
include/treeverify.h carried out request by request, on Python lists and numpy pools.

State: table (B lists of page ids, -1 where none), refs (holders of every page), L (lengths), pools
{m: (K, V)} with K, V [n_pool, P // m, d] for m = 1 (raw), 4 and 128, and optionally keys
[B, c4_cap, d_idx].  Every function changes the state in place and returns the status code.
"""

OK, ERR_ARG, ERR_CAPACITY = 0, -1, -4


def _free(refs):
    return [p for p, r in enumerate(refs) if r == 0]


def _copy(pools, src, dst, tokens):
    for m, (K, V) in pools.items():
        K[dst, :tokens // m] = K[src, :tokens // m]
        V[dst, :tokens // m] = V[src, :tokens // m]


def fork(state, P, source, keep=None):
    table, refs, L, pools = state["table"], state["refs"], state["L"], state["pools"]
    B, G = len(table), len(table[0])
    codes, plan = [], []
    for b in range(B):
        s = source[b]
        if s == -1:
            plan.append(("release", 0, None))
            continue
        if not 0 <= s < B or source[s] != s:
            codes.append(ERR_ARG)
            plan.append(None)
            continue
        kept = [k for k in ((keep[s], keep[b]) if keep is not None else ()) if k >= 0]
        length = min([L[s]] + kept)
        if s == b and length == L[s]:
            plan.append(None)
        elif not 0 <= L[s] <= G * P:
            codes.append(ERR_CAPACITY)
            plan.append(None)
        elif any(not 0 <= p < len(refs) for p in table[s][:-(-length // P)]):
            codes.append(ERR_ARG)
            plan.append(None)
        else:
            plan.append(("truncate" if s == b else "fork", length, s))
    before = [list(row) for row in table]
    shared_before = list(refs)
    counts = list(refs)
    for b, what in enumerate(plan):      # entries that go, full pages that gain a holder
        if what is None:
            continue
        kind, length, s = what
        first = -(-length // P) if kind == "truncate" else 0
        for g in range(first, G):
            if 0 <= before[b][g] < len(refs):
                counts[before[b][g]] -= 1
        if kind == "fork":
            for g in range(length // P):
                counts[before[s][g]] += 1
    wanting = []
    for b, what in enumerate(plan):
        if what is not None and what[1] % P:
            kind, length, s = what
            if kind == "fork" or shared_before[before[s][length // P]] > 1:
                wanting.append(b)
    free = _free(counts)
    if len(wanting) > len(free):
        return ERR_CAPACITY
    refs[:] = counts
    new = dict(zip(wanting, free))
    jobs = []
    for b, what in enumerate(plan):
        if what is None:
            continue
        kind, length, s = what
        full = length // P
        row = [-1] * G
        if kind == "release":
            table[b], L[b] = row, 0
            continue
        row[:full] = before[s][:full]
        if length % P:
            old = before[s][full]
            row[full] = new.get(b, old)
            if b in new:
                refs[new[b]] = 1
                refs[old] -= 1 if kind == "truncate" else 0
                jobs.append((old, new[b], length % P))
        table[b] = row
        L[b] = length
        if kind == "fork" and state.get("keys") is not None:
            state["keys"][b, :length // 4] = state["keys"][s, :length // 4]
    for src, dst, tokens in jobs:
        _copy(pools, src, dst, tokens)
    return codes[0] if codes else OK


def reserve(state, P, need):
    table, refs, L = state["table"], state["refs"], state["L"]
    B, G = len(table), len(table[0])
    codes, want = [], []
    for b in range(B):
        if need[b] <= 0:
            continue
        if L[b] < 0:
            codes.append(ERR_ARG)
        elif L[b] + need[b] > G * P:
            codes.append(ERR_CAPACITY)
        else:
            for g in range(L[b] // P, (L[b] + need[b] - 1) // P + 1):
                if table[b][g] == -1:
                    want.append((b, g))
                elif not 0 <= table[b][g] < len(refs):
                    codes.append(ERR_ARG)
    free = _free(refs)
    if len(want) > len(free):
        return ERR_CAPACITY
    for (b, g), p in zip(want, free):
        table[b][g] = p
        refs[p] = 1
    return codes[0] if codes else OK


def compact(state, P):
    """Returns (code, remap, n_live)."""
    table, refs, L, pools = state["table"], state["refs"], state["L"], state["pools"]
    n, code = len(refs), OK
    tokens, holders = [0] * n, [0] * n
    for b, row in enumerate(table):
        for g, p in enumerate(row):
            if 0 <= p < n:
                tokens[p] = max(tokens[p], min(P, max(0, L[b] - g * P)))
                holders[p] += 1
            elif p != -1:
                code = ERR_ARG
    live = [p for p in range(n) if refs[p] > 0 or holders[p] > 0]
    if any(refs[p] < holders[p] for p in range(n)):
        code = ERR_ARG
    src = [p for p in live if p >= len(live)]
    dst = [p for p in range(len(live)) if p not in set(live)]
    to = {p: p for p in live}
    to.update(zip(src, dst))
    for s, t in zip(src, dst):
        _copy(pools, s, t, P if refs[s] > holders[s] else tokens[s])
        refs[t], refs[s] = refs[s], 0
    for row in table:
        row[:] = [to[p] if 0 <= p < n else p for p in row]
    return code, [to.get(p, -1) for p in range(n)], len(live)
