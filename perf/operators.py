"""What a decode loop does between two verify rounds, as timed and compared cases.

Three operators, each in two forms behind ``run``:

* ``logprobs``: from the logits of a round's tree nodes, per node the natural-log sum of
  exponentials, the entropy, the target token (the largest logit, ties to the lowest id), the K
  best alternatives with their log probabilities, and the log probabilities of given tokens on
  given nodes (a draft tree: every draft token under its parent node).
* ``branch``: the page pool of a batch when requests branch: slots are released, other slots become
  copies of a source slot (its full pages shared by reference count, its last partial page and
  its indexer keys copied), and every slot gets the pages of its next round.
* ``compact``: the live pages of a fragmented pool move into its lowest pages, with the page table
  and the reference counts following.

With ``own`` false, ``run`` computes them in elementary torch operations (fp32); with ``own`` true
it calls this package.  Sizes: 32000 is the package's vocabulary; B = 64 with D = 8 nodes, 512-wide
bf16 rows and 64-wide indexer keys are its serving and long-context workloads; the others are
generic.
"""

import math
import random

import numpy as np
import torch

own = False

_I32 = torch.int32
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one request decoding without speculation: a single row, latency only
        dict(name="logprobs one row", op="logprobs", B=1, D=1, V=32000, pad=0, dtype="bf16", K=1,
             tokens=1, scale=1.0, masked=0),
        # a draft tree growing by one level for one request: few rows, many alternatives each
        dict(name="logprobs draft level", op="logprobs", B=1, D=6, V=200000, pad=0, dtype="f32",
             K=32, tokens=6, scale=1.0, masked=0),
        # the serving batch's verify round
        dict(name="logprobs serving", op="logprobs", B=64, D=8, V=32000, pad=0, dtype="bf16", K=8,
             tokens=8, scale=1.0, masked=0),
        # an odd vocabulary whose rows start at odd elements, a temperature, a vocabulary mask
        dict(name="logprobs odd rows masked", op="logprobs", B=24, D=5, V=50001, pad=2,
             dtype="bf16", K=5, tokens=7, scale=1.25, masked=1),
        # fp32 logits of a larger vocabulary
        dict(name="logprobs wide fp32", op="logprobs", B=32, D=8, V=128000, pad=0, dtype="f32",
             K=20, tokens=8, scale=0.7, masked=0),
        # scoring the given tokens of long texts: many rows, one token each
        dict(name="logprobs scoring", op="logprobs", B=4000, D=1, V=65536, pad=0, dtype="bf16",
             K=0, tokens=1, scale=1.0, masked=0),
        # two prompts sampled four ways each
        dict(name="branch two prompts", op="branch", B=8, ways=4, P=512, lo=200, hi=1500, D=5,
             d=512, dtype="bf16", keys=0, salt=1),
        # a serving batch of which every fourth request survives and branches again
        dict(name="branch serving", op="branch", B=64, ways=4, P=1024, lo=1024, hi=8192, D=8,
             d=512, dtype="bf16", keys=0, salt=2),
        # long contexts with the sparse path's indexer keys
        dict(name="branch long sparse", op="branch", B=32, ways=4, P=2048, lo=30000, hi=65000, D=8,
             d=512, dtype="bf16", keys=64, salt=3),
        # a small pool after a few requests ended
        dict(name="compact small", op="compact", B=8, P=512, lo=200, hi=2500, d=512, dtype="bf16",
             moved=0.25, salt=4),
        # the serving batch's pool
        dict(name="compact serving", op="compact", B=64, P=1024, lo=1024, hi=8192, d=512,
             dtype="bf16", moved=0.3, salt=5),
        # a large pool, half of whose live pages move
        dict(name="compact large", op="compact", B=256, P=512, lo=1024, hi=8192, d=512,
             dtype="bf16", moved=0.5, salt=6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "branch", "compact"])
    if op == "logprobs":
        dtype = rng.choice(["bf16", "f32"])
        V = _log_int(rng, 1000, 260000)
        D = rng.choice([1, 2, 4, 5, 6, 8, 16, 33, 64])
        rows = max(1, min(_log_int(rng, 1, 4000), 500_000_000 // (V * (2 if dtype == "bf16" else 4))))
        return dict(op=op, B=max(1, rows // D), D=D, V=V, pad=rng.choice([0, 0, 1, 8, 63]),
                    dtype=dtype, K=rng.choice([0, 1, 3, 8, 10, 20, 32]),
                    tokens=rng.choice([0, D, rng.randint(1, 100)]),
                    scale=round(rng.uniform(0.5, 2.0), 3), masked=rng.choice([0, 0, 1]))
    dtype, d = rng.choice([("bf16", 512), ("bf16", 512), ("bf16", 72), ("f32", 64), ("f32", 256)])
    P = rng.choice([512, 1024, 1536, 2048])
    B = _log_int(rng, 4, 100)
    lo = rng.randint(1, 3000)
    hi = lo + rng.randint(100, 6000)
    salt = rng.randint(10, 1 << 20)
    if op == "branch":
        return dict(op=op, B=B, ways=rng.randint(2, 8), P=P, lo=lo, hi=hi, D=rng.randint(1, 64),
                    d=d, dtype=dtype, keys=rng.choice([0, 0, 64, 128]), salt=salt)
    return dict(op=op, B=B, P=P, lo=lo, hi=hi, d=d, dtype=dtype,
                moved=round(rng.uniform(0.0, 0.5), 3), salt=salt)


def _lengths(case, n):
    rng = random.Random(case["salt"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(n)]


def _row_bytes(case):
    return case["d"] * (2 if case["dtype"] == "bf16" else 4)


def _layer_rows(tokens):
    """Rows of one page of the three layers that `tokens` valid tokens fill, K and V together."""
    return 2 * (tokens + tokens // 4 + tokens // 128)


def work(case):
    if case["op"] == "logprobs":
        n = case["B"] * case["D"]
        es = 2 if case["dtype"] == "bf16" else 4
        outs = n * (4 + 4 + 4 + 8 * case["K"]) + case["B"] * case["tokens"] * 12
        # per logit: subtract, scale, exponential, two sums
        return {"bytes": n * case["V"] * es + outs, "flops": 6 * n * case["V"]}
    P = case["P"]
    if case["op"] == "branch":
        groups = -(-case["B"] // case["ways"])
        total = meta = 0
        for i, L in enumerate(_lengths(case, groups)):
            forks = min(case["ways"], case["B"] - i * case["ways"]) - 1
            total += forks * 2 * (_layer_rows(L % P) * _row_bytes(case)
                                  + (L // 4) * case["keys"] * 2)
            meta += (forks + 1) * 4 * (2 * (-(-L // P)) + 4)
        return {"bytes": total + meta, "flops": 0}
    c = _compact_plan(case)
    # any live page is as likely to move as any other
    move = c["moved"] / max(1, c["live"]) * sum(_layer_rows(t) for t in c["tokens"]) * _row_bytes(case)
    return {"bytes": 2 * move + 4 * (2 * c["entries"] + 3 * c["pool"]), "flops": 0}


# ---- inputs ------------------------------------------------------------------------------------
def _compact_plan(case):
    """Counts of a compaction case: the requests' lengths, the live pages with their tokens, how
    many of them lie above the live count, and the pool's size.  Every fourth request shares the
    full pages of the one before it."""
    P, B = case["P"], case["B"]
    lengths = _lengths(case, B)
    pages, table, tokens = 0, [], []
    for b, L in enumerate(lengths):
        n = -(-L // P)
        row = list(range(pages, pages + n))
        if b % 4 == 3:
            shared = min(L, lengths[b - 1]) // P
            row = table[b - 1][:shared] + list(range(pages, pages + n - shared))
        fresh = [p for p in row if p >= pages]
        first = n - len(fresh)
        tokens += [min(P, L - (first + i) * P) for i in range(len(fresh))]
        pages += len(fresh)
        table.append(row)
    moved = int(case["moved"] * pages)
    return dict(lengths=lengths, table=table, tokens=tokens, live=pages, moved=moved,
                pool=pages + moved + max(2, pages // 8), entries=sum(len(r) for r in table),
                most=max(len(r) for r in table))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pools(case, n_pool, gen):
    dt, P, d = _TYPES[case["dtype"]], case["P"], case["d"]
    out = {}
    for name, rows in (("rawK", P), ("rawV", P), ("c4K", P // 4), ("c4V", P // 4),
                       ("c128K", P // 128), ("c128V", P // 128)):
        out[name] = torch.empty((n_pool, rows, d), dtype=dt, device="cuda").normal_(generator=gen)
    return out


def _ints(rows):
    return torch.tensor(rows, dtype=_I32).cuda()


def prepare(case, seed):
    gen, rng = _gen(seed), random.Random(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, gen, rng)
    st = _prepare_branch(case, gen, rng) if case["op"] == "branch" else _prepare_compact(case, gen, rng)
    st["case"] = case
    st["status"] = torch.zeros(1, dtype=_I32, device="cuda")
    if own:
        import tree_speculative_verify_gb300 as tv
        n_pool, G, P = st["refs"].numel(), st["table"].shape[1], case["P"]
        st["shape"] = tv.make_shape(
            B=case["B"], D=case.get("D", 1), H=1, d=case["d"],
            dtype=tv.TV_BF16 if case["dtype"] == "bf16" else tv.TV_F32, raw_cap=G * P,
            c4_cap=G * P // 4, c128_cap=G * P // 128, page_tokens=P, max_pages=G,
            n_pool_pages=n_pool, page_table=st["table"])
        st["workspace"] = torch.empty(tv.tv_pages_workspace_size(st["shape"]), dtype=torch.uint8,
                                      device="cuda")
    return st


def _prepare_logprobs(case, gen, rng):
    B, D, V, K, n = case["B"], case["D"], case["V"], case["K"], case["tokens"]
    dt = _TYPES[case["dtype"]]
    store = torch.empty((B, D, V + case["pad"]), dtype=dt, device="cuda")
    store.normal_(generator=gen)
    store *= 2.5
    logits = store[:, :, :V]
    # a few likely tokens per row, as a trained model gives
    likely = torch.randint(0, V, (B, D, 4), generator=gen, device="cuda")
    boost = torch.rand((B, D, 4), generator=gen, device="cuda") * 10 + 4
    logits.scatter_(2, likely, boost.to(dt))
    if case["masked"]:
        # a grammar's mask: a third of the rows keep every 97th token, one row keeps none
        keep = torch.arange(V, device="cuda") % 97 == 0
        rows = torch.arange(B * D, device="cuda").reshape(B, D, 1) % 3 == 1
        logits.masked_fill_(rows & ~keep, -math.inf)
        logits[B - 1, D - 1] = -math.inf
    parents = [[-1] + [rng.randint(0, v - 1) for v in range(1, n)] for _ in range(B)]
    nodes = torch.tensor(parents, dtype=torch.int64).reshape(B, n).remainder_(max(D, 1)) if n else \
        torch.zeros((B, 0), dtype=torch.int64)
    if n > 1:
        nodes[:, 0] = -1       # the root has no parent
    elif n:
        nodes[:, 0] = 0
    nodes = nodes.to(_I32).cuda()
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=_I32)
    if n:
        # every other given token is one of its node's likely ones
        at = likely[torch.arange(B, device="cuda")[:, None], nodes.long().clamp(min=0), 0]
        odd = torch.arange(n, device="cuda") % 2 == 0
        tokens = torch.where(odd, at.to(_I32), tokens)
    f = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")
    i = lambda *s: torch.empty(s, dtype=_I32, device="cuda")
    st = dict(case=case, logits=logits, tokens=tokens, nodes=nodes, lse=f(B, D), entropy=f(B, D),
              logprobs=f(B, n), top_ids=i(B, D, K), top_logprobs=f(B, D, K), target=i(B, D),
              status=torch.zeros(1, dtype=_I32, device="cuda"))
    if own:
        import tree_speculative_verify_gb300 as tv
        st["shape"] = tv.make_shape(B=B, D=D, H=1, d=8, comp_mask=tv.TV_COMP_C4)
    return st


def _prepare_branch(case, gen, rng):
    """Groups of `ways` slots: the first survives, the others hold an earlier branch of their own
    and become copies of it."""
    B, P, ways, D = case["B"], case["P"], case["ways"], case["D"]
    groups = -(-B // ways)
    lengths = _lengths(case, groups)
    rng.shuffle(lengths)
    G = max(-(-(L + D) // P) for L in lengths) + 1
    need = sum(-(-(L + D) // P) for L in lengths) + B * (2 + D // P)
    n_pool = need + sum(1 for b in range(B) if b % ways) + 4
    ids = list(range(n_pool))
    rng.shuffle(ids)
    table, L, source = [], [], []
    for b in range(B):
        if b % ways == 0:
            L.append(lengths[b // ways])
            n = -(-L[-1] // P)
        else:
            L.append(rng.randint(1, P))
            n = 1
        table.append([ids.pop() for _ in range(n)] + [-1] * (G - n))
        source.append(b - b % ways)
    refs = [0] * n_pool
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    st = dict(table=_ints(table), refs=_ints(refs), L=_ints(L), source=_ints(source),
              need=torch.full((B,), D, dtype=_I32, device="cuda"), keys=None)
    st.update(_pools(case, n_pool, gen))
    if case["keys"]:
        st["keys"] = torch.empty((B, G * P // 4, case["keys"]), dtype=torch.bfloat16,
                                 device="cuda").normal_(generator=gen)
    return st


def _prepare_compact(case, gen, rng):
    c = _compact_plan(case)
    n_pool, live, moved = c["pool"], c["live"], c["moved"]
    low = rng.sample(range(live), live - moved)
    high = rng.sample(range(live, n_pool), moved)
    ids = low + high
    rng.shuffle(ids)
    table = [[ids[p] for p in row] + [-1] * (c["most"] + 1 - len(row)) for row in c["table"]]
    refs = [0] * n_pool
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    st = dict(table0=_ints(table), refs0=_ints(refs), L=_ints(c["lengths"]))
    st["table"], st["refs"] = st["table0"].clone(), st["refs0"].clone()
    st["remap"] = torch.empty(n_pool, dtype=_I32, device="cuda")
    st["n_live"] = torch.empty(1, dtype=_I32, device="cuda")
    st.update(_pools(case, n_pool, gen))
    return st


# ---- one pass ----------------------------------------------------------------------------------
_POOLS = ("rawK", "rawV", "c4K", "c4V", "c128K", "c128V")


def run(st):
    op = st["case"]["op"]
    if op == "logprobs":
        return _own_logprobs(st) if own else _plain_logprobs(st)
    if op == "branch":
        return _own_branch(st) if own else _plain_branch(st)
    return _own_compact(st) if own else _plain_compact(st)


def _own_logprobs(st):
    import tree_speculative_verify_gb300 as tv
    tv.tv_token_logprobs(st["shape"], st["logits"], st["tokens"], st["nodes"], st["case"]["scale"],
                         st["lse"], st["entropy"], st["logprobs"], st["top_ids"],
                         st["top_logprobs"], st["target"], st["status"])
    return {k: st[k] for k in ("lse", "entropy", "logprobs", "top_ids", "top_logprobs", "target")}


def _own_branch(st):
    import tree_speculative_verify_gb300 as tv
    pools = [st[k] for k in _POOLS]
    tv.tv_pages_fork(st["shape"], st["source"], None, st["L"], st["refs"], *pools, st["keys"],
                     st["workspace"], st["status"])
    tv.tv_pages_reserve(st["shape"], st["need"], st["L"], st["refs"], st["workspace"], st["status"])
    return _pages_out(st, st["table"], st["refs"], st["L"])


def _own_compact(st):
    import tree_speculative_verify_gb300 as tv
    st["table"].copy_(st["table0"])     # the pool as fragmented as before the last pass
    st["refs"].copy_(st["refs0"])
    tv.tv_pages_compact(st["shape"], st["L"], st["refs"], *[st[k] for k in _POOLS], st["remap"],
                        st["n_live"], st["workspace"], st["status"])
    return dict(_pages_out(st, st["table"], st["refs"], st["L"]), remap=st["remap"],
                n_live=st["n_live"])


def _pages_out(st, table, refs, L):
    out = dict(table=table, refs=refs, L=L)
    for k in _POOLS:
        out[k] = st[k]
    if st.get("keys") is not None:
        out["keys"] = st["keys"]
    return out


def _plain_logprobs(st):
    case = st["case"]
    K, scale = case["K"], case["scale"]
    x = st["logits"].float()
    V = x.shape[2]
    m = x.amax(2, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    y = (x - m0) * scale
    e = y.exp()
    S = e.sum(2, keepdim=True)
    T = torch.where(e > 0, y * e, torch.zeros_like(y)).sum(2, keepdim=True)
    empty = S == 0
    logS = S.log()
    lse = (m * scale + logS)[..., 0]
    entropy = torch.where(empty, torch.zeros_like(S), logS - T / S)[..., 0]
    # alternatives: unique keys in the logits' order, equal logits in the order of their ids
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = order * (1 << 32) + (V - 1 - torch.arange(V, device=x.device))
    ids = torch.topk(key, max(K, 1), dim=2).indices
    value = x.gather(2, ids)
    none = value == -math.inf
    top = torch.where(none, value, (value - m0) * scale - logS)
    ids = torch.where(none, torch.full_like(ids, -1), ids).to(_I32)
    # given tokens
    node = st["nodes"].long()
    b = torch.arange(x.shape[0], device=x.device)[:, None]
    at = node.clamp(min=0)
    given = x[b, at, st["tokens"].long()]
    lp = torch.where(given == -math.inf, given, (given - m0[b, at, 0]) * scale - logS[b, at, 0])
    lp = torch.where(node < 0, torch.zeros_like(lp), lp)
    return dict(lse=lse, entropy=entropy, logprobs=lp, top_ids=ids[..., :K],
                top_logprobs=top[..., :K], target=ids[..., 0])


def _copy_rows(st, src, dst, tokens):
    """Pages src -> dst: the rows that `tokens` valid tokens of each page fill, in every layer."""
    for k, m in zip(_POOLS, (1, 1, 4, 4, 128, 128)):
        pool = st[k]
        rows = torch.arange(pool.shape[1], device=pool.device)[None, :, None]
        pool[dst] = torch.where(rows < (tokens // m)[:, None, None], pool[src], pool[dst])


def _free_ids(refs):
    return torch.sort((refs != 0).to(_I32), stable=True).indices


def _plain_branch(st):
    case = st["case"]
    P = case["P"]
    table, refs, L = st["table"].long(), st["refs"].long(), st["L"].long()
    B, G = table.shape
    s = st["source"].long()
    b, g = torch.arange(B, device=s.device), torch.arange(G, device=s.device)[None]
    forked = s != b
    at = s.clamp(min=0)
    Ln = torch.where(forked, L[at], L)
    # the forked slots' old pages go, the sources' full pages gain a holder each
    old = forked[:, None] & (table >= 0)
    full = forked[:, None] & (g < (Ln // P)[:, None])
    origin = table[at]
    refs = refs.scatter_add(0, table.clamp(min=0).reshape(-1), -old.long().reshape(-1))
    refs = refs.scatter_add(0, origin.clamp(min=0).reshape(-1), full.long().reshape(-1))
    # a new page for each forked slot's partial last page
    tail = forked & (Ln % P > 0)
    new = _free_ids(refs)[(tail.long().cumsum(0) - 1).clamp(min=0)]
    refs = refs.scatter_add(0, new, tail.long())
    mine = torch.where(full, origin, torch.full_like(table, -1))
    mine = torch.where(tail[:, None] & (g == (Ln // P)[:, None]), new[:, None], mine)
    table = torch.where(forked[:, None], mine, table)
    j = tail.nonzero()[:, 0]
    _copy_rows(st, origin[j, Ln[j] // P], new[j], Ln[j] % P)
    if st["keys"] is not None:
        keys = st["keys"]
        j = forked.nonzero()[:, 0]
        rows = torch.arange(keys.shape[1], device=keys.device)[None, :, None]
        keys[j] = torch.where(rows < (Ln[j] // 4)[:, None, None], keys[s[j]], keys[j])
    # the pages of the next round's tokens
    last = (Ln + case["D"] - 1) // P
    want = (g >= (Ln // P)[:, None]) & (g <= last[:, None]) & (table < 0)
    rank = want.long().reshape(-1).cumsum(0) - 1
    new = _free_ids(refs)[rank.clamp(min=0)]
    refs = refs.scatter_add(0, new, want.long().reshape(-1))
    table = torch.where(want, new.reshape(B, G), table)
    return _pages_out(st, table.to(_I32), refs.to(_I32), Ln.to(_I32))


def _plain_compact(st):
    P = st["case"]["P"]
    table, refs, L = st["table0"].long(), st["refs0"].long(), st["L"].long()
    n_pool, G = refs.numel(), table.shape[1]
    ids = torch.arange(n_pool, device=refs.device)
    mapped = table >= 0
    page = table.clamp(min=0).reshape(-1)
    # tokens of every page; a page that somebody besides the table holds counts as full
    held = (L[:, None] - P * torch.arange(G, device=L.device)).clamp(0, P)
    tokens = torch.zeros_like(refs).scatter_reduce(
        0, page, torch.where(mapped, held, torch.zeros_like(held)).reshape(-1), "amax")
    holders = torch.zeros_like(refs).scatter_add(0, page, mapped.long().reshape(-1))
    tokens = torch.where(refs > holders, torch.full_like(tokens, P), tokens)
    live = (refs > 0) | (holders > 0)
    n_live = live.long().sum()
    src = (live & (ids >= n_live)).nonzero()[:, 0]
    dst = (~live & (ids < n_live)).nonzero()[:, 0]
    remap = torch.where(live, ids, torch.full_like(ids, -1))
    remap[src] = dst
    _copy_rows(st, src, dst, tokens[src])
    new_refs = torch.zeros_like(refs)
    new_refs[remap[live]] = refs[live]
    table = torch.where(mapped, remap[table.clamp(min=0)], table)
    return dict(_pages_out(st, table.to(_I32), new_refs.to(_I32), st["L"]), remap=remap.to(_I32),
                n_live=n_live.to(_I32).reshape(1))


# ---- the definitions in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(case, st)
    return _exact_branch(case, st) if case["op"] == "branch" else _exact_compact(case, st)


def _exact_logprobs(case, st):
    B, D, V, scale, n = case["B"], case["D"], case["V"], case["scale"], case["tokens"]
    lse, entropy = np.full((B, D), -np.inf), np.zeros((B, D))
    lp = np.zeros((B, n))
    nodes, tokens = st["nodes"].cpu().numpy(), st["tokens"].cpu().numpy()
    top = np.full((B, D, case["K"]), -np.inf)
    step = max(1, 100_000_000 // (D * V))
    for lo in range(0, B, step):
        z = st["logits"][lo:lo + step].double() * float(np.float32(scale))
        total = torch.logsumexp(z, 2)
        logp = z - total[..., None]
        p = logp.exp()
        h = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(2)
        some = torch.isfinite(total)
        lse[lo:lo + step] = total.cpu().numpy()
        entropy[lo:lo + step] = torch.where(some, h, torch.zeros_like(h)).cpu().numpy()
        best = torch.topk(z, case["K"], dim=2).values - total[..., None]
        best = torch.where(some[..., None], best, torch.full_like(best, -math.inf))
        top[lo:lo + step] = best.cpu().numpy()
        if n:
            nd = torch.as_tensor(nodes[lo:lo + step]).long().cuda()
            tk = torch.as_tensor(tokens[lo:lo + step]).long().cuda()
            i = torch.arange(nd.shape[0], device="cuda")[:, None].expand_as(nd)
            row = nd.clamp(min=0)
            v = torch.where(some[i, row], logp[i, row, tk], torch.full_like(z[i, row, tk], -math.inf))
            lp[lo:lo + step] = torch.where(nd < 0, torch.zeros_like(v), v).cpu().numpy()
    return dict(lse=lse, entropy=entropy, logprobs=lp, top_ids=None, top_logprobs=top, target=None)


def _move(st, jobs):
    for src, dst, tokens in jobs:
        for k, m in (("rawK", 1), ("rawV", 1), ("c4K", 4), ("c4V", 4), ("c128K", 128), ("c128V", 128)):
            st[k][dst, :tokens // m] = st[k][src, :tokens // m]


def _exact_branch(case, st):
    P, B = case["P"], case["B"]
    table, refs, L = st["table"].tolist(), st["refs"].tolist(), st["L"].tolist()
    source = st["source"].tolist()
    G = len(table[0])
    for b in range(B):
        if source[b] != b:
            for p in table[b]:
                if p >= 0:
                    refs[p] -= 1
            s = source[b]
            L[b] = L[s]
            table[b] = [table[s][g] if g < L[b] // P else -1 for g in range(G)]
            for g in range(L[b] // P):
                refs[table[b][g]] += 1
    free = lambda: next(p for p in range(len(refs)) if refs[p] == 0)
    jobs = []
    for b in range(B):
        if source[b] != b and L[b] % P:
            g, p = L[b] // P, free()
            refs[p], table[b][g] = 1, p
            jobs.append((table[source[b]][g], p, L[b] % P))
    for b in range(B):
        for g in range(L[b] // P, (L[b] + case["D"] - 1) // P + 1):
            if table[b][g] < 0:
                table[b][g] = free()
                refs[table[b][g]] = 1
    _move(st, jobs)
    if st["keys"] is not None:
        for b in range(B):
            st["keys"][b, :L[b] // 4] = st["keys"][source[b], :L[b] // 4].clone()
    return _pages_out(st, _ints(table), _ints(refs), _ints(L))


def _exact_compact(case, st):
    P = case["P"]
    table, refs, L = st["table0"].tolist(), st["refs0"].tolist(), st["L"].tolist()
    tokens, n_pool = {}, len(refs)
    for b, row in enumerate(table):
        for g, p in enumerate(row):
            if p >= 0:
                tokens[p] = max(tokens.get(p, 0), min(P, max(0, L[b] - g * P)))
    live = [p for p in range(n_pool) if refs[p] > 0]
    n = len(live)
    src = [p for p in live if p >= n]
    dst = [p for p in range(n) if refs[p] == 0]
    to = {p: p for p in live}
    to.update(zip(src, dst))
    _move(st, [(s, t, tokens.get(s, P)) for s, t in zip(src, dst)])
    table = [[to[p] if p >= 0 else -1 for p in row] for row in table]
    new = [0] * n_pool
    for p in live:
        new[to[p]] = refs[p]
    return dict(_pages_out(st, _ints(table), _ints(new), _ints(L)),
                remap=_ints([to.get(p, -1) for p in range(n_pool)]), n_live=_ints([n]))
