"""How new tokens come into the compressed cache and how beams go on, as timed and compared cases.

Three operators, each in two forms behind ``run``:

* ``append``: the new tokens of a ragged batch (a prompt, a part of one, one token per request) go
  behind the committed ones: the last ``rope`` dimensions of their keys are rotated by their
  position, keys and values are stored in their cache rows (contiguous or in pages), the C4 and C128
  entry of every block that they complete is written, the lengths advance; their queries, where
  given, are rotated too.
* ``attend``: the queries of such a chunk over the cache that now holds it: a token at position p
  sees the C4 entries below p // 4, the C128 entries below p // 128 and the raw rows p - W .. p.
* ``beam``: from the logits of the beams of every group and their scores the best continuations, in
  the slots that the cache's pages are then reordered by.

With ``own`` false, ``run`` computes them in elementary torch operations (fp32, angles and scores next
to each other in fp64); with ``own`` true it calls this package.  Sizes: 64 requests of 1024 to 8192
tokens, 64 heads on one 512-wide bf16 key and value, a window of 128, pages of 1024 tokens and a
vocabulary of 32000 are the package's serving workload, 65536 tokens its long context, fp32 rows of 64
with 8 heads its smallest; the others are generic.
"""

import math
import random

import torch

own = False

_I32 = torch.int32
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one request decoding: its newest token goes into the cache, latency only
        dict(name="append one token", op="append", B=1, H=64, d=512, dtype="bf16", rope=64,
             pairs=1, P=0, lo=1000, hi=1000, new="one", most=1, salt=1),
        # one token of every request of the serving batch, the cache in pages
        dict(name="append serving step", op="append", B=64, H=64, d=512, dtype="bf16", rope=64,
             pairs=1, P=1024, lo=1024, hi=8192, new="one", most=1, salt=2),
        # prompts of very different lengths behind short prefixes, the smallest rows, no queries
        dict(name="append ragged fp32", op="append", B=13, H=0, d=64, dtype="f32", rope=64,
             pairs=0, P=0, lo=0, hi=300, new="mixed", most=1500, salt=3),
        # a long prompt with its queries
        dict(name="append prompt", op="append", B=1, H=64, d=512, dtype="bf16", rope=64, pairs=0,
             P=1024, lo=0, hi=0, new="all", most=16384, salt=4),
        # one request decoding at 8192 tokens, latency
        dict(name="attend one token", op="attend", B=1, H=64, d=512, dtype="bf16", P=1024, W=128,
             lo=8192, hi=8192, new="one", most=1, salt=5),
        # the serving batch, one token per request
        dict(name="attend serving step", op="attend", B=64, H=64, d=512, dtype="bf16", P=1024,
             W=128, lo=1024, hi=8192, new="one", most=1, salt=6),
        # a step that mixes decoding requests with parts of prompts, odd sizes
        dict(name="attend mixed step", op="attend", B=24, H=64, d=512, dtype="bf16", P=1024, W=100,
             lo=0, hi=6000, new="mixed", most=777, salt=7),
        # the package's smallest rows in fp32
        dict(name="attend ragged fp32", op="attend", B=6, H=8, d=64, dtype="f32", P=0, W=128, lo=0,
             hi=2000, new="mixed", most=400, salt=8),
        # the next part of a prompt that is already 65536 tokens long
        dict(name="attend long prompt", op="attend", B=1, H=64, d=512, dtype="bf16", P=2048, W=128,
             lo=65536, hi=65536, new="all", most=1024, salt=9),
        # four beams of one request
        dict(name="beam one request", op="beam", G=1, width=4, V=32000, pad=0, dtype="bf16",
             scale=1.0, masked=0, first=0, ended=0.0),
        # eight beams of 64 requests, some of them ended
        dict(name="beam serving", op="beam", G=64, width=8, V=32000, pad=0, dtype="bf16",
             scale=1.0, masked=0, first=0, ended=0.2),
        # wide beams over a larger odd vocabulary in fp32 with a grammar's mask
        dict(name="beam wide fp32", op="beam", G=16, width=16, V=128001, pad=2, dtype="f32",
             scale=0.8125, masked=1, first=0, ended=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "beam"])
    salt = rng.randint(10, 1 << 20)
    if op == "beam":
        dtype, width = rng.choice(["bf16", "f32"]), rng.choice([1, 2, 3, 4, 5, 8, 10, 16, 32])
        V = _log_int(rng, 1000, 200000)
        rows = max(1, min(_log_int(rng, 1, 600), 120_000_000 // (V * (2 if dtype == "bf16" else 4))))
        return dict(op=op, G=max(1, rows // width), width=width, V=V, pad=rng.choice([0, 0, 1, 8, 63]),
                    dtype=dtype, scale=rng.randint(32, 128) / 64, masked=rng.choice([0, 0, 1]),
                    first=rng.choice([0, 0, 0, 1]), ended=rng.choice([0.0, 0.0, 0.3]))
    dtype, d = rng.choice([("bf16", 512)] * 5 + [("bf16", 128), ("f32", 64), ("f32", 256)])
    H = rng.choice([64, 64, 64, 32, 128, 24]) if d == 512 else rng.choice([4, 8, 16, 11])
    new = rng.choice(["one", "mixed", "all"])
    B = _log_int(rng, 1, 100) if new == "one" else _log_int(rng, 1, 24)
    lo = rng.choice([0, rng.randint(0, 3000), rng.randint(0, 20000)])
    hi = lo + rng.randint(0, 4000)
    most = 1 if new == "one" else _log_int(rng, 2, 2000 if d == 512 else 500)
    B = max(1, min(B, 500_000 // (hi + 1)))
    case = dict(op=op, B=B, H=H, d=d, dtype=dtype, P=rng.choice([0, 512, 1024, 1536]), lo=lo, hi=hi,
                new=new, most=most, salt=salt)
    if op == "append":
        case.update(H=rng.choice([0, H]), rope=rng.choice([0, 64, min(d, 128)]),
                    pairs=rng.choice([0, 1]))
    else:
        case.update(W=rng.choice([0, 37, 128, 128, 300]))
    while True:     # at most what the largest listed cases cost
        w = work(case)
        if w["bytes"] <= 1_500_000_000 and w["flops"] <= (2e12 if d == 512 else 1e11):
            return case
        case["most" if case["most"] > 1 else "B"] //= 2


def _sizes(case):
    """Committed lengths before the chunk and new tokens of every request, whole batch."""
    rng = random.Random(case["salt"])
    before = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["new"] == "mixed":      # mostly single tokens, some requests without any, some parts
        news = [rng.choice([1, 1, 1, 0, rng.randint(1, case["most"]), rng.randint(1, case["most"])])
                for _ in range(case["B"])]
        news[0] = max(1, case["most"])
    else:
        news = [case["most"]] * case["B"]
    return before, news


def _closing(before, news, m):
    """Rows that were committed before and belong to blocks of m that the new tokens complete, and
    the blocks completed."""
    rows = blocks = 0
    for L, n in zip(before, news):
        k = (L + n) // m - L // m
        blocks += k
        rows += L % m if k else 0
    return rows, blocks


def _seen(p, W):
    return p // 4 + p // 128 + min(p, W) + 1


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "beam":
        rows = case["G"] * case["width"]
        return {"bytes": rows * (case["V"] * es + 28), "flops": 6 * rows * case["V"]}
    before, news = _sizes(case)
    n, d, H = sum(news), case["d"], case["H"]
    if case["op"] == "append":
        old4, new4 = _closing(before, news, 4)
        old128, new128 = _closing(before, news, 128)
        rows = 4 * n + 2 * max(old4, old128) + 2 * (new4 + new128) + 2 * n * H
        return {"bytes": rows * d * es, "flops": n * (12 * d + 3 * case["rope"] * (1 + H))}
    flops = rows = 0
    for L, k in zip(before, news):
        flops += 4 * d * H * sum(_seen(p, case["W"]) for p in range(L, L + k))
        if k:
            last = L + k - 1
            rows += 2 * (last // 4 + last // 128 + last + 1 - max(0, L - case["W"]))
    return {"bytes": rows * d * es + 2 * n * H * d * es + 4 * n * H, "flops": flops}


# ---- inputs ------------------------------------------------------------------------------------
_POOLS = ("rawK", "rawV", "c4K", "c4V", "c128K", "c128V")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = _prepare_beam(case, gen) if case["op"] == "beam" else _prepare_cache(case, gen, seed)
    st["case"] = case
    st["status"] = torch.zeros(1, dtype=_I32, device="cuda")
    if own:
        import tree_speculative_verify_gb300 as tv
        if case["op"] == "beam":
            st["shape"] = tv.make_shape(B=case["G"] * case["width"], D=1, H=1, d=8,
                                        comp_mask=tv.TV_COMP_C4)
            size = tv.tv_beam_workspace_size(st["shape"], case["width"])
        else:
            P, cap = case["P"], st["cap"]
            paged = {}
            if P:
                paged = dict(page_tokens=P, max_pages=cap // P, n_pool_pages=st["rawK"].shape[0],
                             page_table=st["table"])
            st["shape"] = tv.make_shape(
                B=case["B"], D=1, H=max(1, case["H"]), d=case["d"], W=case.get("W", 128),
                dtype=tv.TV_BF16 if case["dtype"] == "bf16" else tv.TV_F32, raw_cap=cap,
                c4_cap=cap // 4, c128_cap=cap // 128, **paged)
            size = 0
            if case["op"] == "attend":
                size = tv.tv_chunk_workspace_size(st["shape"], st["n"])
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return st


def _prepare_cache(case, gen, seed):
    """A cache of `before` tokens per request, and the chunk; for `attend` the chunk lies in it."""
    B, H, d, P = case["B"], case["H"], case["d"], case["P"]
    dt = _TYPES[case["dtype"]]
    before, news = _sizes(case)
    most = max(L + n for L, n in zip(before, news))
    unit = P if P else 128
    G = -(-(most + 1) // unit)
    cap = G * unit
    if P:
        ids = list(range(B * G + 3))
        random.Random(seed).shuffle(ids)
        table = torch.tensor(ids[:B * G], dtype=_I32).reshape(B, G).cuda()
        sizes = [(len(ids), P // m, d) for m in (1, 1, 4, 4, 128, 128)]
    else:
        table = None
        sizes = [(B, cap // m, d) for m in (1, 1, 4, 4, 128, 128)]
    st = dict(table=table, cap=cap, before=before, news=news, n=sum(news))
    # compressed entries are averages of raw rows and smaller than they are
    for name, size, std in zip(_POOLS, sizes, (0.5, 0.5, 0.35, 0.35, 0.2, 0.2)):
        st[name] = torch.empty(size, dtype=dt, device="cuda").normal_(0.0, std, generator=gen)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    st["starts"] = torch.tensor(starts, dtype=_I32).cuda()
    normal = lambda std, *s: torch.empty(s, dtype=dt, device="cuda").normal_(0.0, std, generator=gen)
    n = st["n"]
    if case["op"] == "append":
        st["L0"] = torch.tensor(before, dtype=_I32).cuda()
        st["L"] = st["L0"].clone()
        st["K"], st["V"] = normal(0.5, n, d), normal(0.5, n, d)
        st["Q"] = normal(1.0, n, H, d) if H else None
        st["Qr"] = torch.empty_like(st["Q"]) if H else None
        st["g4"] = torch.empty(d, device="cuda").normal_(generator=gen)
        st["g128"] = torch.empty(d, device="cuda").normal_(generator=gen)
        half = case["rope"] // 2
        i = torch.arange(half, dtype=torch.float64)
        st["inv_freq"] = (10000.0 ** (-i / max(half, 1))).float().cuda() if half else None
    else:
        st["L"] = torch.tensor([L + k for L, k in zip(before, news)], dtype=_I32).cuda()
        # queries that single some keys out, as a trained model's do
        st["Q"] = normal(3.0 * math.sqrt(512.0 / d), n, H, d)
        st["O"] = torch.empty_like(st["Q"])
        st["lse"] = torch.empty((n, H), dtype=torch.float32, device="cuda")
    return st


def _prepare_beam(case, gen):
    G, W, V = case["G"], case["width"], case["V"]
    B = G * W
    dt = _TYPES[case["dtype"]]
    store = torch.empty((B, V + case["pad"]), dtype=dt, device="cuda")
    store.normal_(generator=gen)
    store *= 2.5
    logits = store[:, :V]
    likely = torch.randint(0, V, (B, 6), generator=gen, device="cuda")
    boost = torch.rand((B, 6), generator=gen, device="cuda") * 8 + 6
    logits.scatter_(1, likely, boost.to(dt))
    row = torch.arange(B, device="cuda")[:, None]
    if case["masked"]:
        # a grammar's mask: a third of the rows keep every 97th token, one beam's row keeps none
        keep = torch.arange(V, device="cuda") % 97 == 0
        logits.masked_fill_((row % 3 == 1) & ~keep, -math.inf)
        logits[B - 1] = -math.inf
    scores = -torch.rand(B, generator=gen, device="cuda") * 6 - 20
    if case["first"]:       # a group's first step: one beam that counts
        scores[row[:, 0] % W != 0] = -math.inf
    done = (torch.rand(B, generator=gen, device="cuda") < case["ended"]).to(_I32)
    i = lambda: torch.empty(B, dtype=_I32, device="cuda")
    return dict(logits=logits, scores=scores, done=done, source=i(), token=i(), rank=i(),
                new_done=i(), new_scores=torch.empty(B, dtype=torch.float32, device="cuda"), eos=2)


# ---- one pass ----------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if op == "append":
        return _own_append(st) if own else _plain_append(st)
    if op == "attend":
        return _own_attend(st) if own else _plain_attend(st)
    return _own_beam(st) if own else _plain_beam(st)


def _append_out(st):
    out = {k: st[k] for k in _POOLS + ("L",)}
    if st["Qr"] is not None:
        out["Qr"] = st["Qr"]
    return out


def _own_append(st):
    import tree_speculative_verify_gb300 as tv
    st["L"].copy_(st["L0"])     # as many tokens as before the last pass
    tv.tv_chunk_append(st["shape"], st["starts"], st["K"], st["V"], st["Q"], st["case"]["rope"],
                       st["case"]["pairs"], st["inv_freq"], st["g4"], st["g128"], st["Qr"],
                       *[st[k] for k in _POOLS], st["L"], st["status"])
    return _append_out(st)


def _own_attend(st):
    import tree_speculative_verify_gb300 as tv
    tv.tv_chunk_attn(st["shape"], st["starts"], st["Q"], st["c4K"], st["c4V"], st["c128K"],
                     st["c128V"], st["rawK"], st["rawV"], st["L"], 1.0 / math.sqrt(st["case"]["d"]),
                     st["O"], st["lse"], st["workspace"], st["status"])
    return dict(O=st["O"], lse=st["lse"])


def _own_beam(st):
    import tree_speculative_verify_gb300 as tv
    tv.tv_beam_select(st["shape"], st["case"]["width"], st["logits"], st["scores"], st["done"],
                      st["eos"], st["case"]["scale"], st["source"], st["token"], st["new_scores"],
                      st["new_done"], st["rank"], st["workspace"], st["status"])
    return {k: st[k] for k in ("source", "token", "new_scores", "new_done", "rank")}


def _rows(st, b, row, m):
    """Row of row `row` of request `b` in a layer of one row per m tokens, flat over the layer."""
    if st["table"] is None:
        return b * (st["cap"] // m) + row
    per = st["case"]["P"] // m
    return st["table"].long()[b, row // per] * per + row % per


def _token_index(st):
    """Request and place in its chunk of every new token."""
    news = (st["starts"][1:] - st["starts"][:-1]).long()
    B = news.numel()
    b = torch.repeat_interleave(torch.arange(B, device=news.device), news, output_size=st["n"])
    return b, torch.arange(st["n"], device=news.device) - st["starts"].long()[b]


def _rotate(x, angle, rope, pairs):
    """The last `rope` values of x's rows (fp32) as pairs rotated by angle [..., rope / 2]."""
    if not rope:
        return x
    x = x.clone()
    tail = x[..., -rope:]
    if pairs:
        a, c = tail[..., 0::2].clone(), tail[..., 1::2].clone()
    else:
        a, c = tail[..., :rope // 2].clone(), tail[..., rope // 2:].clone()
    cos, sin = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    first, second = a * cos - c * sin, a * sin + c * cos
    if pairs:
        tail[..., 0::2], tail[..., 1::2] = first, second
    else:
        tail[..., :rope // 2], tail[..., rope // 2:] = first, second
    return x


def _plain_append(st):
    case = st["case"]
    dt, d, rope = st["K"].dtype, case["d"], case["rope"]
    st["L"].copy_(st["L0"])
    b, i = _token_index(st)
    pos = st["L"].long()[b] + i
    angle = None
    if rope:      # in fp64: an angle of 65536 radians in fp32 is off by 0.004
        angle = pos.double()[:, None] * st["inv_freq"].double()[None]
    flat = {k: st[k].reshape(-1, d) for k in _POOLS}
    at = _rows(st, b, pos, 1)
    flat["rawK"][at] = _rotate(st["K"].float(), angle, rope, case["pairs"]).to(dt)
    flat["rawV"][at] = st["V"]
    for m, g, K, V in ((4, "g4", "c4K", "c4V"), (128, "g128", "c128K", "c128V")):
        end = ((pos + 1) % m == 0).nonzero()[:, 0]
        for part in end.split(8192):
            first = pos[part] + 1 - m
            block = _rows(st, b[part][:, None], first[:, None] + torch.arange(m, device=at.device), 1)
            rk, rv = flat["rawK"][block].float(), flat["rawV"][block].float()
            z = (rk * st[g]).sum(2)
            w = (z - z.amax(1, keepdim=True)).exp()
            w = (w / w.sum(1, keepdim=True))[..., None]
            to = _rows(st, b[part], first // m, m)
            flat[K][to], flat[V][to] = (w * rk).sum(1).to(dt), (w * rv).sum(1).to(dt)
    if st["Q"] is not None:
        for lo in range(0, st["n"], 2048):
            cut = slice(lo, lo + 2048)
            turn = None if angle is None else angle[cut, None]
            st["Qr"][cut] = _rotate(st["Q"][cut].float(), turn, rope, case["pairs"]).to(dt)
    st["L"] += (st["starts"][1:] - st["starts"][:-1])
    return _append_out(st)


def _plain_attend(st):
    case = st["case"]
    W, H, d = case["W"], case["H"], case["d"]
    scale = 1.0 / math.sqrt(d)
    dev = st["Q"].device
    flat = {k: st[k].reshape(-1, d) for k in _POOLS}
    start = 0
    for b, (L, n) in enumerate(zip(st["before"], st["news"])):
        if n == 0:
            continue
        lo, last = max(0, L - W), L + n - 1
        n4, n128 = last // 4, last // 128
        every = [(n4, "c4", 4, 0), (n128, "c128", 128, 0), (last + 1 - lo, "raw", 1, lo)]
        K, V, key = [], [], []
        for count, name, m, first in every:
            row = first + torch.arange(count, device=dev)
            at = _rows(st, b, row, m)
            K.append(flat[name + "K"][at].float())
            V.append(flat[name + "V"][at].float())
            # a row is seen by positions key <= p; a raw row also only by p <= position + W
            key.append(row if m == 1 else m * (row + 1))
        K, V, key = torch.cat(K), torch.cat(V), torch.cat(key)
        raw = torch.arange(key.numel(), device=dev) >= n4 + n128
        step = max(1, 400_000_000 // (H * key.numel()))
        for t in range(0, n, step):
            k = min(step, n - t)
            p = L + t + torch.arange(k, device=dev)
            q = st["Q"][start + t:start + t + k].reshape(k * H, d).float()
            s = ((q @ K.T) * scale).reshape(k, H, -1)
            seen = (key[None] <= p[:, None]) & (~raw[None] | (key[None] >= p[:, None] - W))
            s = s.masked_fill_(~seen[:, None], -math.inf)
            top = s.amax(2, keepdim=True)
            e = s.sub_(top).exp_()
            total = e.sum(2, keepdim=True)
            o = (e.reshape(k * H, -1) @ V).reshape(k, H, d) / total
            st["O"][start + t:start + t + k] = o.to(st["O"].dtype)
            st["lse"][start + t:start + t + k] = (top + total.log())[..., 0]
        start += n
    return dict(O=st["O"], lse=st["lse"])


def _plain_beam(st):
    case = st["case"]
    G, W, V = case["G"], case["width"], case["V"]
    x = st["logits"].float()
    # candidates of a beam: its W largest logits, equal ones in the order of their ids
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = order * (1 << 32) + (V - 1 - torch.arange(V, device=x.device))
    ids = torch.topk(key, W, dim=1).indices
    # scores of different beams may lie next to each other: in fp64
    y = x.double() * case["scale"]
    top = y.amax(1, keepdim=True)
    some = top > -math.inf
    top = torch.where(some, top, torch.zeros_like(top))
    lse = top + (y - top).exp().sum(1, keepdim=True).log()
    lp = torch.where(some, y.gather(1, ids) - lse, torch.full_like(ids, -math.inf, dtype=torch.float64))
    ended = st["done"][:, None] != 0
    lp = torch.where(ended, torch.full_like(lp, -math.inf), lp)
    lp[:, 0] = torch.where(ended[:, 0], torch.zeros_like(lp[:, 0]), lp[:, 0])
    ids = torch.where(ended, torch.full_like(ids, st["eos"]), ids)
    total = (st["scores"].double()[:, None] + lp).reshape(G, -1)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :W], at[:, :W]
    alive = best > -math.inf
    beam = at // W
    token = ids.reshape(G, -1).gather(1, at)
    # a beam's best continuation stays in its slot, the others fill the free slots in order
    same = (beam[:, :, None] == beam[:, None, :]).tril(-1)
    stays = alive & ~same.any(2)
    taken = torch.zeros((G, W), dtype=torch.int64, device=x.device)
    taken.scatter_add_(1, beam, stays.long())
    free = torch.sort(taken, dim=1, stable=True).indices
    slot = torch.where(stays, beam, free.gather(1, ((~stays).long().cumsum(1) - 1).clamp(min=0)))
    base = torch.arange(G, device=x.device)[:, None] * W
    none = torch.full_like(token, -1)
    rank = torch.arange(W, device=x.device).expand(G, W)
    was = st["done"].long().reshape(G, W).gather(1, beam)
    over = alive & ((was != 0) | (token == st["eos"]))

    def put(values, dtype):
        out = torch.empty((G, W), dtype=dtype, device=x.device)
        return out.scatter_(1, slot, values.to(dtype)).reshape(-1)

    return dict(source=put(torch.where(alive, base + beam, none), _I32),
                token=put(torch.where(alive, token, none), _I32),
                new_scores=put(best, torch.float32), new_done=put(over, _I32),
                rank=put(torch.where(alive, rank, none), _I32))


# ---- the definitions in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_attend(case, st) if case["op"] == "attend" else _exact_beam(case, st)


def _page_row(st, b, row, m):
    if st["table"] is None:
        return b, row
    per = st["case"]["P"] // m
    return int(st["pages"][b][row // per]), row % per


def _turn(x, positions, case, freq):
    """Rotation by complex numbers: pairs (a, c) as a + ic times exp(i p f)."""
    rope = case["rope"]
    x = x.double()
    if not rope:
        return x
    tail = x[..., x.shape[-1] - rope:]
    both = tail.unflatten(-1, (rope // 2, 2)) if case["pairs"] else \
        tail.unflatten(-1, (2, rope // 2)).transpose(-1, -2)
    z = torch.complex(both[..., 0], both[..., 1])
    turn = torch.polar(torch.ones_like(freq)[None], positions.double()[:, None] * freq[None])
    while turn.dim() < z.dim():
        turn = turn[:, None]
    z = torch.view_as_real(z * turn)
    tail = z.flatten(-2) if case["pairs"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([x[..., :x.shape[-1] - rope], tail], -1)


def _exact_append(case, st):
    st["case"] = case
    if st["table"] is not None:
        st["pages"] = st["table"].tolist()
    out = {k: st[k].double() for k in _POOLS}
    stored = {k: st[k].clone() for k in ("rawK", "rawV")}
    freq = None if st["inv_freq"] is None else st["inv_freq"].double()
    start, unit = 0, case["P"] or st["cap"]
    Qr = None if st["Q"] is None else torch.empty(st["Q"].shape, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(st["before"], st["news"])):
        pos = torch.arange(L, L + n, device="cuda")
        K = _turn(st["K"][start:start + n], pos, case, freq)
        V = st["V"][start:start + n].double()
        for lo in range(0, n, 1024) if Qr is not None else ():
            hi = min(n, lo + 1024)
            Qr[start + lo:start + hi] = _turn(st["Q"][start + lo:start + hi], pos[lo:hi], case, freq)
        t = 0
        while t < n:        # page by page
            k = min(n - t, unit - (L + t) % unit)
            page, row = _page_row(st, b, L + t, 1)
            for name, x in (("rawK", K), ("rawV", V)):
                out[name][page, row:row + k] = x[t:t + k]
                stored[name][page, row:row + k] = x[t:t + k].to(stored[name].dtype)
            t += k
        for m, g, c in ((4, st["g4"], "c4"), (128, st["g128"], "c128")):
            first, end = L // m, (L + n) // m
            while first < end:      # the entries of one page, from the rows as they are stored
                k = min(end - first, (unit - (first * m) % unit) // m)
                page, row = _page_row(st, b, first * m, 1)
                to, j = _page_row(st, b, first, m)
                kk = stored["rawK"][page, row:row + k * m].double().reshape(k, m, -1)
                vv = stored["rawV"][page, row:row + k * m].double().reshape(k, m, -1)
                w = torch.softmax(kk @ g.double(), 1)[:, None]
                out[c + "K"][to, j:j + k] = (w @ kk)[:, 0]
                out[c + "V"][to, j:j + k] = (w @ vv)[:, 0]
                first += k
        start += n
    out["L"] = torch.tensor([L + n for L, n in zip(st["before"], st["news"])], dtype=_I32)
    if Qr is not None:
        out["Qr"] = Qr
    return out


def _exact_attend(case, st):
    W, H, d = case["W"], case["H"], case["d"]
    if work(case)["flops"] > 6e12:
        return None
    O = torch.empty(st["O"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device="cuda")
    start = 0

    def layer(name, b, count, m):
        if st["table"] is None:
            return st[name][b, :count].double()
        per = case["P"] // m
        pages = st["table"][b, :-(-count // per)].long()
        return st[name][pages].reshape(-1, d)[:count].double()

    for b, (L, n) in enumerate(zip(st["before"], st["news"])):
        if n == 0:
            continue
        total = L + n
        ends = [torch.arange(1, total // m + 1, device="cuda") * m for m in (4, 128)]
        raw = torch.arange(max(0, L - W), total, device="cuda")
        K = torch.cat([layer("c4K", b, total // 4, 4), layer("c128K", b, total // 128, 128),
                       layer("rawK", b, total, 1)[raw]])
        V = torch.cat([layer("c4V", b, total // 4, 4), layer("c128V", b, total // 128, 128),
                       layer("rawV", b, total, 1)[raw]])
        # the positions that see a row: from `begin` up to `until`
        begin = torch.cat(ends + [raw])
        until = torch.cat([torch.full_like(e, 1 << 40) for e in ends] + [raw + W])
        step = max(1, 100_000_000 // (H * begin.numel()))
        for t in range(0, n, step):
            k = min(step, n - t)
            p = torch.arange(L + t, L + t + k, device="cuda")[:, None, None]
            z = torch.einsum("thd,nd->thn", st["Q"][start + t:start + t + k].double(), K) / math.sqrt(d)
            z = torch.where((p >= begin) & (p <= until), z, torch.full_like(z, -math.inf))
            lse[start + t:start + t + k] = torch.logsumexp(z, 2)
            O[start + t:start + t + k] = torch.softmax(z, 2) @ V
        start += n
    return dict(O=O, lse=lse)


def _exact_beam(case, st):
    G, W, V = case["G"], case["width"], case["V"]
    scores, done = st["scores"].double().tolist(), st["done"].tolist()
    result = {k: [None] * (G * W) for k in ("source", "token", "new_scores", "new_done", "rank")}
    for g in range(G):
        lines = list(range(g * W, g * W + W))
        logp = torch.log_softmax(st["logits"][g * W:g * W + W].double() * case["scale"], 1)
        logp = torch.where(logp.isnan(), torch.full_like(logp, -math.inf), logp)
        best, ids = torch.sort(logp, dim=1, descending=True, stable=True)
        best, ids = best[:, :W].tolist(), ids[:, :W].tolist()
        found = []
        for w, b in enumerate(lines):
            if done[b]:
                found.append((-scores[b], w, st["eos"], 1))
            else:
                found += [(-scores[b] - lp, w, x, int(x == st["eos"])) for lp, x in zip(best[w], ids[w])]
        found = sorted(f for f in found if f[0] < math.inf)[:W]
        slots, rest = {}, []
        for k, f in enumerate(found):
            if f[1] in slots:
                rest.append(k)
            else:
                slots[f[1]] = k
        free = [w for w in range(W) if w not in slots]
        slots.update(zip(free, rest))
        for w, b in enumerate(lines):
            k = slots.get(w, -1)
            value = (-1, -1, -math.inf, 0, -1) if k < 0 else (
                g * W + found[k][1], found[k][2], -found[k][0], found[k][3], k)
            for name, v in zip(("source", "token", "new_scores", "new_done", "rank"), value):
                result[name][b] = v
    out = {k: _ints(v) for k, v in result.items() if k != "new_scores"}
    out["new_scores"] = torch.tensor(result["new_scores"], dtype=torch.float64)
    return out


def _ints(values):
    return torch.tensor(values, dtype=_I32).cuda()
