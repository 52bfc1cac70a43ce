"""tv_pages_fork, tv_pages_reserve and tv_pages_compact on the GPU against the oracle: tables, counts,
lengths and every row of every pool exactly, over worked cases and random histories; and a decode
loop on a managed pool against the same rounds on contiguous caches."""

import copy
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import pages
from tree_speculative_verify_gb300 import _lib, engine, workloads

pytestmark = pytest.mark.gpu

MS = {1: ("rawK", "rawV"), 4: ("c4K", "c4V"), 128: ("c128K", "c128V")}


class Pool:
    """One state on the GPU and its copy for the oracle."""

    def __init__(self, table, L, n_pool, P=512, d=8, dtype="bf16", comp=(4, 128), extra=(), keys=0,
                 seed=0, ws_spare=0):
        B, G = len(table), len(table[0])
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator().manual_seed(seed)
        self.P, self.comp = P, comp
        self.t = {}
        for m in (1,) + tuple(comp):
            for name in MS[m]:
                self.t[name] = torch.randn((n_pool, P // m, d), generator=g).to(dt).cuda()
        refs = [0] * n_pool
        for row in table:
            for p in row:
                if 0 <= p < n_pool:
                    refs[p] += 1
        for p in extra:
            refs[p] += 1
        i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
        self.table, self.refs, self.L, self.status = i32(table), i32(refs), i32(L), i32([0])
        self.keys = torch.randn((B, G * P // 4, keys), generator=g).bfloat16().cuda() if keys else None
        mask = (_lib.TV_COMP_C4 if 4 in comp else 0) | (_lib.TV_COMP_C128 if 128 in comp else 0)
        self.shape = _lib.make_shape(
            B=B, D=8, H=1, d=d, comp_mask=mask, dtype=_lib.TV_BF16 if dtype == "bf16" else _lib.TV_F32,
            raw_cap=G * P, c4_cap=G * P // 4, c128_cap=G * P // 128, page_tokens=P, max_pages=G,
            n_pool_pages=n_pool, page_table=self.table)
        self.ws = torch.full((_lib.tv_pages_workspace_size(self.shape) + ws_spare,), 0x5a,
                             dtype=torch.uint8, device="cuda")
        self.remap = torch.full((n_pool,), -9, dtype=torch.int32, device="cuda")
        self.n_live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        self.o = dict(table=[list(r) for r in table], refs=refs, L=list(L),
                      pools={m: tuple(self.np(self.t[k]) for k in MS[m]) for m in (1,) + tuple(comp)},
                      keys=self.np(self.keys) if keys else None)

    @staticmethod
    def np(t):
        return t.float().cpu().numpy()

    def layers(self):
        return [self.t.get(k) for m in (1, 4, 128) for k in MS[m]]

    def fork(self, source, keep=None, stream=None):
        i32 = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32).cuda()
        s, k = i32(source), i32(keep)
        torch.cuda.synchronize()
        _lib.tv_pages_fork(self.shape, s, k, self.L, self.refs, *self.layers(), self.keys, self.ws,
                           self.status, stream)
        torch.cuda.synchronize()
        return pages.fork(self.o, self.P, list(source), None if keep is None else list(keep))

    def reserve(self, need):
        _lib.tv_pages_reserve(self.shape, torch.tensor(need, dtype=torch.int32).cuda(), self.L,
                              self.refs, self.ws, self.status)
        return pages.reserve(self.o, self.P, list(need))

    def compact(self):
        _lib.tv_pages_compact(self.shape, self.L, self.refs, *self.layers(), self.remap, self.n_live,
                              self.ws, self.status)
        code, remap, n = pages.compact(self.o, self.P)
        assert self.remap.tolist() == remap and self.n_live.tolist() == [n]
        return code

    def check(self, codes):
        """`codes`: what the oracle returned, in order; the status word holds one of the errors."""
        torch.cuda.synchronize()
        assert self.table.tolist() == self.o["table"]
        assert self.refs.tolist() == self.o["refs"]
        assert self.L.tolist() == self.o["L"]
        for m, pools in self.o["pools"].items():
            for k, want in zip(MS[m], pools):
                assert np.array_equal(self.np(self.t[k]), want), k
        if self.keys is not None:
            assert np.array_equal(self.np(self.keys), self.o["keys"])
        status = int(self.status.item())
        errors = [c for c in codes if c]
        assert (status in (-1, -4)) if errors else status == 0
        if errors and all(c == errors[0] for c in errors):
            assert status == errors[0]
        self.status.zero_()


def _random_table(rng, B, G, n_pool, L, P):
    ids = list(rng.permutation(n_pool))
    return [[int(ids.pop()) for _ in range(-(-n // P))] + [-1] * (G - -(-n // P)) for n in L]


@pytest.mark.parametrize("d,dtype,comp,keys", [(8, "bf16", (4, 128), 0), (512, "bf16", (4, 128), 64),
                                               (24, "f32", (4,), 8), (72, "bf16", (128,), 0)])
@pytest.mark.parametrize("P", [512, 1536])
def test_fork_copies_shares_and_releases(P, d, dtype, comp, keys):
    rng = np.random.default_rng(P + d)
    L = [0, 1, 3, P - 1, P, P + 1, 2 * P, 2 * P + 127, 2 * P + 300, 5]
    s = Pool(_random_table(rng, 10, 4, 40, L, P), L, 40, P, d, dtype, comp, keys=keys)
    codes = [s.fork([0, 1, 2, 3, 4, 5, 6, 7, 8, 9])]                   # nothing to do
    codes.append(s.fork([0, 0, 2, 3, 3, 5, 6, 8, 8, 8]))               # empty, partial, many of one
    s.check(codes)
    codes = [s.fork([0, 1, 2, -1, -1, 5, 6, 6, -1, 5])]                # release and fork together
    s.check(codes)
    codes = [s.fork([0, 1, 2, 5, 6, 5, 6, 6, 8, 5], [-1, -1, 2, 9, P + 1, 1, -1, P, -1, 2000])]
    s.check(codes)


def test_fork_refuses_slots_one_by_one():
    P = 512
    L = [700, 40, 600, 1100, 5, 2000, 9]
    table = [[0, 1, -1], [2, -1, -1], [3, -1, -1], [4, 5, 6], [7, -1, -1], [8, 9, 10], [77, -1, -1]]
    s = Pool(table, L, 16, P)
    # out of range; source that moves; source with a missing page; source past the capacity; a
    # page outside the pool; two good ones
    s.check([s.fork([0, 9, 2, 2, 3, 5, 5])])
    s.check([s.fork([0, -2, 2, 0, 6, 5, 6])])
    s.check([s.fork([0, 0, 2, 3, 4, 5, 0])])


def test_one_page_too_few_leaves_everything():
    P = 512
    s = Pool([[0, 1], [2, -1], [3, -1], [-1, -1]], [600, 10, 20, 0], 5, P, ws_spare=64)
    s.check([s.fork([0, 0, 2, 0])])            # released page 2 and free page 4: just enough
    s.check([s.reserve([0, 0, 500, 0])])       # no page missing but one: none is free
    s.check([s.fork([0, 0, 0, 0])])            # the copies take the released pages
    s.check([s.fork([0, 1, -1, 3]), s.reserve([P, 0, 5, 0])])
    s.check([s.fork([0, 1, 0, 3])])


def test_truncation_copies_a_page_that_others_hold():
    P = 512
    s = Pool([[0, 1, 2], [-1] * 3, [-1] * 3], [1200, 0, 0], 10, P)
    s.check([s.fork([0, 0, 0])])
    s.check([s.fork([0, 1, 2], [100, 1024, 1200])])   # into a shared page, to its end, not at all
    s.check([s.fork([0, 1, 2], [-1, 600, 600])])      # two holders of one page at once
    s.check([s.fork([0, 1, 2], [0, 512, 99999])])


def test_reserve_windows():
    P = 512
    rng = np.random.default_rng(4)
    L = [0, 511, 512, 505, 100, 1023, 2000]
    s = Pool(_random_table(rng, 7, 6, 40, L, P), L, 40, P)
    s.check([s.reserve([1, 1, 8, 8, 0, 2000, -3])])
    s.check([s.reserve([8] * 7)])
    s.check([s.reserve([0, 3000, 1, 0, 0, 0, 1072])])   # one past the capacity, one to its end
    s.L[2] = -4
    s.o["L"][2] = -4
    s.check([s.reserve([8] * 7)])


@pytest.mark.parametrize("n_pool,B,G", [(3, 1, 2), (40, 6, 5), (700, 50, 8), (5000, 300, 6), (8193, 300, 6),
                                        (700, 50, 800)])
def test_compact_moves_the_upper_live_pages(n_pool, B, G):
    P, rng = 512, np.random.default_rng(n_pool)
    L = [int(x) for x in rng.integers(0, min(G, 8) * P + 1, size=B)]
    while sum(-(-n // P) for n in L) > 0.8 * n_pool:
        L[int(np.argmax(L))] = int(rng.integers(0, 2 * P))
    table = _random_table(rng, B, G, n_pool, L, P)
    for b in range(2, B, 3):                            # some share their first full pages
        for g in range(min(L[b], L[b - 1]) // P):
            table[b][g] = table[b - 1][g]
    held = {p for r in table for p in r}
    extra = [p for p in range(n_pool - 1, 0, -5)][:40]   # pages that others hold too, or alone
    s = Pool(table, L, n_pool, P, extra=extra)
    assert s.compact() == 0
    s.check([])
    assert int(s.n_live) == len((held | set(extra)) - {-1})
    assert s.compact() == 0                              # nothing is left to move
    s.check([])
    assert s.remap.tolist()[:int(s.n_live)] == list(range(int(s.n_live)))


@pytest.mark.parametrize("n_pool", [400, 9000])
def test_reserve_of_long_prompts(n_pool):
    # windows of many pages, some of them mapped already, beside short ones
    P, G, B = 512, 150, 40
    rng = np.random.default_rng(n_pool)
    L = [int(x) for x in rng.integers(0, 3 * P, size=B)]
    table = _random_table(rng, B, G, 300, L, P)
    for b in (3, 7):
        table[b][9] = 301 + b
    s = Pool(table, L, n_pool, P)
    need = [int(x) for x in rng.integers(1, 9, size=B)]
    need[3], need[5], need[7], need[33], need[39] = 40 * P, 5 * P, 33 * P + 1, 32 * P, 6 * P
    s.check([s.reserve(need)])
    need[3] = 150 * P
    s.check([s.reserve(need)])       # past the capacity, and the others once more: nothing is missing


def test_compact_reports_an_inconsistent_table():
    P = 512
    s = Pool([[5, 90], [3, -1]], [600, 20], 8, P)
    s.refs[5] = 0
    s.o["refs"][5] = 0
    assert s.compact() == -1
    s.check([-1])


@pytest.mark.parametrize("seed,wide", [(0, 0), (1, 0), (2, 0), (3, 0), (4, 1), (5, 1)])
def test_random_histories(seed, wide):
    # (wide: a table of more entries than one CTA plans, so that the cluster does)
    rng = np.random.default_rng(seed)
    B, G, P, n = int(rng.integers(3, 40)), int(rng.integers(2, 7)), 512, 90
    if wide:
        G = 40000 // B
    s = Pool([[-1] * G for _ in range(B)], [0] * B, n, P, keys=16, seed=seed)
    for _ in range(25):
        op, codes = int(rng.integers(4)), []
        if op <= 1:
            need = [int(x) for x in rng.integers(-20, 700, size=B)]
            codes.append(s.reserve(need))
            for b in range(B):     # a round's commit: the length moves where the pages are there
                new = s.o["L"][b] + max(0, need[b])
                if new <= G * P and -1 not in s.o["table"][b][:-(-new // P)]:
                    s.o["L"][b] = new
            s.L.copy_(torch.tensor(s.o["L"], dtype=torch.int32))
        elif op == 2:
            src = [int(x) if rng.random() < 0.4 else b for b, x in enumerate(rng.integers(-1, B, size=B))]
            keep = [int(x) for x in rng.integers(-900, min(G, 7) * P, size=B)] if rng.random() < 0.5 else None
            codes.append(s.fork(src, keep))
        else:
            codes.append(s.compact())
        s.check(codes)


def test_host_refusals():
    s = Pool([[0, -1]], [5], 4)
    src = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = _lib.make_shape(B=1, D=8, H=1, d=8, raw_cap=1024, c4_cap=256, c128_cap=8)
    for shape, ws, code in ((plain, s.ws, -2), (s.shape, s.ws[:256], -7), (s.shape, None, -1),
                            (s.shape, s.ws[16:], -1)):
        with pytest.raises(_lib.TreeVerifyError) as e:
            _lib.tv_pages_reserve(shape, src, s.L, s.refs, ws, s.status)
        assert e.value.code == code
    with pytest.raises(ValueError):
        _lib.tv_pages_reserve(s.shape, src, s.L, s.refs[:2], s.ws, s.status)
    with pytest.raises(TypeError):
        _lib.tv_pages_fork(s.shape, src.long(), None, s.L, s.refs, *s.layers(), None, s.ws, s.status)
    with pytest.raises(ValueError):
        _lib.tv_pages_fork(s.shape, src, None, s.L, s.refs, s.t["rawK"][:1], *s.layers()[1:], None,
                           s.ws, s.status)
    s.check([])


def test_two_captured_graphs_and_another_stream():
    P = 512
    s = Pool([[3, 4, -1], [5, -1, -1], [-1] * 3], [700, 30, 0], 12, P)
    src = torch.tensor([0, 1, 0], dtype=torch.int32).cuda()
    drop = torch.tensor([0, 1, -1], dtype=torch.int32).cuda()
    need = torch.tensor([8, 8, 400], dtype=torch.int32).cuda()
    graphs = []
    for a in (src, drop):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.tv_pages_fork(s.shape, a, None, s.L, s.refs, *s.layers(), None, s.ws, s.status)
            _lib.tv_pages_reserve(s.shape, need, s.L, s.refs, s.ws, s.status)
            _lib.tv_pages_compact(s.shape, s.L, s.refs, *s.layers(), s.remap, s.n_live, s.ws, s.status)
        graphs.append(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in (0, 1, 0, 1):
        with torch.cuda.stream(side):
            graphs[k].replay()
        torch.cuda.synchronize()
        pages.fork(s.o, P, (src, drop)[k].tolist())
        pages.reserve(s.o, P, need.tolist())
        pages.compact(s.o, P)
        s.check([])


def _commit_rows(wl, seed, n):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn((wl.B, wl.D, wl.d), generator=g) * 0.5).to(wl.torch_dtype).cuda()
            for _ in range(2 * n)]


@pytest.mark.parametrize("kernel,stage", [(_lib.TV_ATTN_AUTO, 0), (_lib.TV_ATTN_SIMT, 0), (_lib.TV_ATTN_AUTO, 1)])
def test_decode_loop_on_a_managed_pool(kernel, stage):
    """Rounds, branching, releasing and compaction on a managed pool, the targets from logits:
    every round's outputs and every request's visible cache equal those of contiguous caches that
    are forked by whole copies."""
    wl = workloads.serving(B=6, L=(500, 1400))
    P = 512
    shape, st = engine.alloc_pool(wl, P, 40, kernel, stage_chain=stage)
    rb = engine.alloc_round(wl, shape)
    engine.alloc_scores(rb, shape, 1000, n_top=3)
    engine.prefill(shape, st, rb)
    cshape = engine.shape_for(wl, kernel, stage_chain=stage)
    cshape.raw_cap, cshape.c4_cap, cshape.c128_cap = shape.raw_cap, shape.c4_cap, shape.c128_cap
    z = lambda rows: torch.zeros((wl.B, rows, wl.d), dtype=wl.torch_dtype, device="cuda")
    cst = engine.DeviceState(rawK=z(shape.raw_cap), rawV=z(shape.raw_cap), c4K=z(shape.c4_cap),
                             c4V=z(shape.c4_cap), c128K=z(shape.c128_cap), c128V=z(shape.c128_cap),
                             L=st.L.clone())
    cst.rawK[:, :wl.raw_cap], cst.rawV[:, :wl.raw_cap] = wl.rawK.cuda(), wl.rawV.cuda()
    crb = engine.alloc_round(wl, cshape)
    engine.prefill(cshape, cst, crb)
    remap = torch.empty(40, dtype=torch.int32, device="cuda")
    n_live = torch.empty(1, dtype=torch.int32, device="cuda")
    rows = _commit_rows(wl, 5, 6)
    steps = [None, [0, 0, 2, 2, 2, 5], None, [0, 1, 4, -1, 4, 0], "compact", None]
    for i, step in enumerate(steps):
        if step == "compact":
            engine.compact(shape, st, rb, remap, n_live)
        elif step is not None:
            engine.fork(shape, st, rb, torch.tensor(step, dtype=torch.int32).cuda())
            for name in ("rawK", "rawV", "c4K", "c4V", "c128K", "c128V", "L"):
                t = getattr(cst, name)
                old = t.clone()
                for b, s in enumerate(step):
                    if s >= 0:
                        t[b] = old[s]
                    elif name == "L":
                        t[b] = 0
        for r in (rb, crb):
            r.treeK.copy_(rows[2 * i])
            r.treeV.copy_(rows[2 * i + 1])
        rb.logits.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
        draft = torch.tensor(wl.draft).cuda().long() % 1000
        # most nodes' best token is their first child's
        first = torch.full((wl.B, wl.D), -1, dtype=torch.long, device="cuda")
        for v in range(wl.D - 1, 0, -1):
            par = rb.parents[:, v].long()
            first.scatter_(1, par[:, None], draft[:, v:v + 1])
        boost = torch.where(first >= 0, 9.0, -9.0)
        rb.logits.scatter_(2, first.clamp(min=0)[..., None], boost[..., None].to(rb.logits.dtype))
        rb.draft.copy_(draft.int())
        crb.draft.copy_(draft.int())
        engine.verify_round(shape, st, rb, scored=True)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        crb.target.copy_(rb.logits.float().argmax(2).int())
        engine.verify_round(cshape, cst, crb)
        torch.cuda.synchronize()
        assert int(crb.status.item()) == 0
        for name in ("target", "accept_len", "path", "bonus", "committed", "O", "lse"):
            assert torch.equal(getattr(rb, name), getattr(crb, name)), (i, name)
        assert torch.equal(st.L, cst.L)
        assert int(rb.accept_len.max()) > 1
        table = st.page_table.long()
        for b in range(wl.B):
            L = int(st.L[b])
            for m, (k, v) in MS.items():
                for name in (k, v):
                    pool = getattr(st, name)
                    got = pool[table[b].clamp(min=0)].reshape(-1, wl.d)[:L // m]
                    assert torch.equal(got, getattr(cst, name)[b, :L // m]), (i, b, name)
    counts = np.bincount(st.page_table.cpu().numpy().ravel() + 1, minlength=41)[1:]
    assert st.page_refs.tolist() == counts[:40].tolist()


def test_round_without_free_pages_commits_nothing_it_has_no_page_for():
    # request 0 ends exactly at its page's end, and no page is free: its commit is refused, the other
    # request's page still has room
    wl = workloads.serving(B=2, L=(512, 512))
    wl.L[1] = 300
    shape, st = engine.alloc_pool(wl, 512, 2)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    before = {k: getattr(st, k).clone() for k in ("rawK", "c4K", "c128K")}
    engine.verify_round(shape, st, rb)
    torch.cuda.synchronize()
    assert int(rb.status.item()) == _lib_code("TV_ERR_CAPACITY")
    assert st.L.tolist() == [512, 300 + int(rb.accept_len[1])]
    assert rb.committed[0].tolist() == [-1] * wl.D
    page = int(st.page_table[0, 0])
    for k, t in before.items():
        assert torch.equal(getattr(st, k)[page], t[page]), k


def _lib_code(name):
    return next(c for c, n in _lib.TV_ERR.items() if n == name)


def test_calls_right_behind_the_acceptance_walk_see_its_results():
    # the walk allows the kernel behind it to start early and stores its results only after the
    # attention in front of it has completed: whatever reads them must have waited for the walk
    wl = workloads.serving(B=40, L=(2048, 2048))
    shape, st = engine.alloc_pool(wl, 512, 400)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    engine.plan(shape, st, rb)
    engine.branch_compress(shape, st, rb)
    logits = torch.randn((40, 1, 40000), generator=torch.Generator(device="cuda").manual_seed(1),
                         device="cuda")
    one = _lib.make_shape(B=40, D=1, H=1, d=8, comp_mask=1)
    lp, lse = (torch.empty((40, 1), device="cuda") for _ in range(2))
    stay = torch.arange(40, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def walk():
        for t in (rb.accept_len, rb.bonus):
            t.zero_()
        torch.cuda.synchronize()
        engine.attention(shape, st, rb)
        engine.accept(shape, st, rb)

    walk()
    engine.reserve(shape, st, rb, need=rb.accept_len)
    torch.cuda.synchronize()
    n = rb.accept_len.clone()
    assert int(rb.status.item()) == 0 and int(n.min()) >= 1
    assert bool((st.page_table[:, 4] >= 0).all())       # position 2048 lies on the fifth page
    walk()
    _lib.tv_token_logprobs(one, logits, rb.bonus.view(40, 1), None, 1.0, lse, None, lp, None, None, None,
                           rb.status)
    torch.cuda.synchronize()
    want = torch.log_softmax(logits.double(), 2).gather(2, rb.bonus.long().view(40, 1, 1))[..., 0]
    assert bool((rb.bonus != 0).any()) and float((lp - want).abs().max()) < 1e-4
    walk()
    engine.fork(shape, st, rb, stay, keep=rb.accept_len)
    torch.cuda.synchronize()
    assert int(rb.status.item()) == 0 and torch.equal(st.L, n)
    refs = torch.bincount((st.page_table[st.page_table >= 0]).long(), minlength=400)
    assert torch.equal(refs.int(), st.page_refs) and int((st.page_table >= 0).sum()) == 40


def test_round_graph_on_a_managed_pool():
    # replayed rounds map their pages, commit and move on like rounds called one by one
    wl = workloads.serving(B=5, L=(500, 900))
    runs = []
    for graphed in (False, True):
        shape, st = engine.alloc_pool(wl, 512, 24)
        rb = engine.alloc_round(wl, shape)
        engine.alloc_scores(rb, shape, workloads.VOCAB, n_top=2)
        engine.prefill(shape, st, rb)
        rb.logits.normal_(generator=torch.Generator(device="cuda").manual_seed(9))
        graph = engine.RoundGraph(shape, st, rb, scored=True) if graphed else None
        for _ in range(8):
            graph.replay() if graphed else engine.verify_round(shape, st, rb, scored=True)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        view = st.page_table.long().clamp(min=0)
        runs.append([st.L, st.page_table, st.page_refs, rb.O, rb.target, rb.top_ids, rb.committed]
                    + [getattr(st, k)[view] for m in MS for k in MS[m]])
    assert int((runs[0][0].cpu() - torch.as_tensor(wl.L)).min()) >= 8
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_branch_on_the_sparse_path_selects_what_its_source_selects():
    # the fork carries the indexer keys: with the same queries, tokens and tree the branch's round is
    # its source's, from the device selection to the committed rows
    wl = workloads.long_context(B=3, L=(9000, 12000), n_sel=512)
    shape, st = engine.alloc_pool(wl, 2048, 24)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    for t in (rb.Q, rb.treeK, rb.treeV, rb.parents, rb.draft, rb.target, rb.q_idx):
        t[2] = t[0]
    before = st.k_idx.clone()
    engine.fork(shape, st, rb, torch.tensor([0, 1, 0], dtype=torch.int32).cuda())
    engine.verify_round(shape, st, rb, select=True)
    torch.cuda.synchronize()
    assert int(rb.status.item()) == 0
    n = int(wl.L[0]) // 4
    assert torch.equal(st.k_idx[2, :n], before[0, :n]) and torch.equal(st.k_idx[2, n:], before[2, n:])
    for name in ("sel", "O", "lse", "accept_len", "path", "bonus", "committed"):
        t = getattr(rb, name)
        assert torch.equal(t[2], t[0]), name
    assert int(st.L[2]) == int(st.L[0]) > int(wl.L[0])
    table = st.page_table.long()
    for m in MS:
        for name in MS[m]:
            rows = [getattr(st, name)[table[b].clamp(min=0)].reshape(-1, wl.d)[:int(st.L[0]) // m] for b in (0, 2)]
            assert torch.equal(*rows), name


def test_calls_on_two_streams_at_once():
    # two pools, each with its own workspace, and two batches of logits, on two streams
    P = 512
    rng = np.random.default_rng(8)
    pools = []
    for k in range(2):
        L = [int(x) for x in rng.integers(1, 3 * P, size=40)]
        pools.append(Pool(_random_table(rng, 40, 5, 400, L, P), L, 400, P, d=64, seed=k))
    x = [torch.randn((1, 30, 60000), generator=torch.Generator(device="cuda").manual_seed(k), device="cuda")
         for k in range(2)]
    f = lambda: torch.empty((1, 30), device="cuda")
    out = [(f(), f(), torch.empty((1, 30, 9), dtype=torch.int32, device="cuda"),
            torch.empty((1, 30, 9), device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    shape = _lib.make_shape(B=1, D=30, H=1, d=8, comp_mask=1)
    src = [[b - b % 3 for b in range(40)], [b - b % 5 for b in range(40)]]
    src_t = [torch.tensor(s, dtype=torch.int32).cuda() for s in src]
    need = torch.full((40,), 700, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for k, s in enumerate(pools):
            st = streams[k]
            _lib.tv_pages_fork(s.shape, src_t[k], None, s.L, s.refs, *s.layers(), None, s.ws, s.status, st)
            _lib.tv_token_logprobs(shape, x[k], None, None, 1.0, out[k][0], out[k][1], None, out[k][2],
                                   out[k][3], None, s.status, st)
            _lib.tv_pages_reserve(s.shape, need, s.L, s.refs, s.ws, s.status, st)
            _lib.tv_pages_compact(s.shape, s.L, s.refs, *s.layers(), s.remap, s.n_live, s.ws, s.status, st)
    torch.cuda.synchronize()
    for k, s in enumerate(pools):
        for _ in range(3):
            codes = [pages.fork(s.o, P, src[k]), pages.reserve(s.o, P, [700] * 40), pages.compact(s.o, P)[0]]
        s.check(codes)
        assert torch.equal(out[k][2], torch.topk(x[k], 9, dim=2).indices.int())


def test_copied_pool_goes_its_own_way():
    # branching, compaction and rounds on one of the two leave the other's rounds as they are
    wl = workloads.serving(B=4, L=(500, 1400))
    shape, st = engine.alloc_pool(wl, 512, 30)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    cshape, copy = engine.clone_pool(shape, st)
    want_shape, want = engine.clone_pool(shape, st)
    wrb, crb = engine.alloc_round(wl, shape), engine.alloc_round(wl, shape)
    engine.verify_round(want_shape, want, wrb)
    remap = torch.empty(30, dtype=torch.int32, device="cuda")
    n_live = torch.empty(1, dtype=torch.int32, device="cuda")
    engine.fork(shape, st, rb, torch.tensor([0, -1, 0, 0], dtype=torch.int32).cuda())
    engine.compact(shape, st, rb, remap, n_live)
    engine.verify_round(shape, st, rb)
    engine.verify_round(cshape, copy, crb)
    torch.cuda.synchronize()
    assert [int(r.status.item()) for r in (rb, wrb, crb)] == [0, 0, 0]
    for name in ("L", "page_table", "page_refs", "rawK", "c4V", "c128K"):
        assert torch.equal(getattr(copy, name), getattr(want, name)), name
    for name in ("O", "lse", "committed"):
        assert torch.equal(getattr(crb, name), getattr(wrb, name)), name
    assert not torch.equal(st.page_table, copy.page_table)


@pytest.mark.parametrize("call", ["fork", "reserve", "compact"])
def test_scratch_pad_right_behind_a_pages_call_sees_its_results(call):
    # no plan between them: the scratch pad reads lengths, page numbers and rows that the call in front
    # writes, and stages rows on pages that it maps
    wl = workloads.serving(B=24, L=(1021, 2046))
    for k in range(6):
        runs = []
        for waits in (True, False):
            shape, st = engine.alloc_pool(wl, 512, 200, stage_chain=1)
            rb = engine.alloc_round(wl, shape)
            engine.prefill(shape, st, rb)
            remap = torch.empty(200, dtype=torch.int32, device="cuda")
            n_live = torch.empty(1, dtype=torch.int32, device="cuda")
            src = torch.arange(24, dtype=torch.int32, device="cuda")
            keep = torch.tensor([509 + 3 * k + b for b in range(24)], dtype=torch.int32, device="cuda")
            if call == "compact":      # two thirds of the slots go, the others' pages move down
                drop = torch.where(src % 3 == 2, src, torch.full_like(src, -1))
                engine.fork(shape, st, rb, drop)
                rb.need.copy_(torch.where(drop >= 0, rb.need, 0))
            if call != "reserve":
                engine.reserve(shape, st, rb)
            torch.cuda.synchronize()
            if call == "fork":
                engine.fork(shape, st, rb, torch.where(src % 4 == 3, src - 3, src), keep)
            elif call == "reserve":
                engine.reserve(shape, st, rb)
            else:
                engine.compact(shape, st, rb, remap, n_live)
            if waits:
                torch.cuda.synchronize()
            engine.branch_compress(shape, st, rb)
            torch.cuda.synchronize()
            live = [b for b in range(24) if call != "compact" or b % 3 == 2]
            table = st.page_table.long().clamp(min=0)
            runs.append([t[live] for t in (rb.scrK4, rb.scrV4, rb.scrK128, rb.scrV128, st.L, st.page_table)]
                        + [st.rawK[table[live]], st.c4K[table[live]]])
        for a, b in zip(*runs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kernel,stage,sparse", [
    (_lib.TV_ATTN_AUTO, 0, False), (_lib.TV_ATTN_AUTO, 1, False), (_lib.TV_ATTN_SIMT, 0, False),
    (_lib.TV_ATTN_AUTO, 0, True), (_lib.TV_ATTN_SIMT, 1, True)])
def test_released_slots_stay_empty(kernel, stage, sparse):
    # rounds, called and replayed, pass over slots without a need: no page, no length, no error, and
    # the others' rounds are those of a batch in which nothing was released
    wl = workloads.long_context(B=4, L=(9000, 12000), n_sel=512) if sparse else \
        workloads.serving(B=5, L=(500, 1400))
    P, n_pool = (2048, 32) if sparse else (512, 24)
    shape, st = engine.alloc_pool(wl, P, n_pool, kernel, stage_chain=stage)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    fshape, full = engine.clone_pool(shape, st)
    frb = engine.alloc_round(wl, fshape)
    gone, live = [1, 3], [b for b in range(wl.B) if b not in (1, 3)]
    source = torch.arange(wl.B, dtype=torch.int32, device="cuda")
    source[gone] = -1
    engine.fork(shape, st, rb, source)
    rb.need[gone] = 0
    free = n_pool - len({p for b in live for p in st.page_table[b].tolist() if p >= 0})
    assert int((st.page_refs == 0).sum()) == free
    graph = None
    for k in range(4):
        if k < 2:
            engine.verify_round(shape, st, rb, select=sparse)
        else:
            graph = graph or engine.RoundGraph(shape, st, rb, select=sparse)
            graph.replay()
        engine.verify_round(fshape, full, frb, select=sparse)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == int(frb.status.item()) == 0
        assert st.L[gone].tolist() == [0, 0]
        assert bool((st.page_table[gone] == -1).all()) and bool((rb.committed[gone] == -1).all())
        held = st.page_table[st.page_table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=n_pool).int(), st.page_refs)
        for name in ("O", "lse", "accept_len", "path", "bonus", "committed"):
            assert torch.equal(getattr(rb, name)[live], getattr(frb, name)[live]), name
        assert torch.equal(st.L[live], full.L[live])
    engine.draft_decode(shape, st, rb)
    torch.cuda.synchronize()
    assert int(rb.status.item()) == 0 and st.L[gone].tolist() == [0, 0]
    if not sparse:
        rb.need[1] = wl.D          # a request starts on the slot
        engine.verify_round(shape, st, rb)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        assert st.L[gone].tolist() == [int(rb.accept_len[1]), 0] and int(st.page_table[1, 0]) >= 0


def test_missing_page_of_a_live_request_is_still_an_error():
    wl = workloads.serving(B=2, L=(512, 512))
    shape, st = engine.alloc_pool(wl, 512, 4)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    rb.need.zero_()
    L = st.L.clone()
    engine.verify_round(shape, st, rb)
    torch.cuda.synchronize()
    assert int(rb.status.item()) == _lib_code("TV_ERR_ARG")
    assert torch.equal(st.L, L) and bool((rb.committed == -1).all())
    # nor is a slot empty whose first page is there, or whose table holds another number
    for first in (2, 77):
        rb.status.zero_()
        st.L.zero_()
        st.page_table.fill_(-1)
        st.page_table[:, 0] = torch.tensor([first, first + 1], dtype=torch.int32)
        engine.verify_round(shape, st, rb)
        torch.cuda.synchronize()
        want = 0 if first == 2 else _lib_code("TV_ERR_ARG")
        assert int(rb.status.item()) == want
        assert (st.L.tolist() == [0, 0]) == (first == 77)


@pytest.mark.parametrize("stage", [0, 1])
def test_capturing_a_round_takes_no_pages(stage):
    # neither with pages to spare nor without, when the capture's own round cannot have its pages
    wl = workloads.serving(B=3, L=(512, 512))
    for n_pool in (3, 12):
        shape, st = engine.alloc_pool(wl, 512, n_pool, stage_chain=stage)
        rb = engine.alloc_round(wl, shape)
        engine.prefill(shape, st, rb)
        torch.cuda.synchronize()
        state = [st.L, st.page_table, st.page_refs, rb.status, st.rawK[:3], st.c4V[:3], st.c128K[:3]]
        before = [t.clone() for t in state]
        shorter = st.L - 10
        graph = engine.RoundGraph(shape, st, rb, prologue=lambda: st.L.copy_(shorter))
        for a, b in zip(state, before):
            assert torch.equal(a, b)
        graph.replay()               # at the prologue's lengths every position has its page
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        assert torch.equal(st.L, shorter + rb.accept_len)
        assert st.page_table[:, 1:].max() == -1 and int(st.page_refs.sum()) == 3


def test_calls_from_two_host_threads():
    # pools of different sizes, both planned by one CTA with more shared memory than a kernel gets
    # unasked: neither thread's launches fail for the other's
    import threading
    P, errors, pools = 512, [], []
    for k, n_pool in enumerate((8192, 6300)):
        L = [700] * 8
        pools.append(Pool([[n_pool - 1 - 2 * b, n_pool - 2 - 2 * b, -1] for b in range(8)], L, n_pool, P, seed=k))
    need = torch.full((8,), 8, dtype=torch.int32, device="cuda")
    stay = torch.arange(8, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def work(s):
        try:
            stream = torch.cuda.Stream()
            for _ in range(2000):
                _lib.tv_pages_fork(s.shape, stay, None, s.L, s.refs, *s.layers(), None, s.ws, s.status, stream)
                _lib.tv_pages_reserve(s.shape, need, s.L, s.refs, s.ws, s.status, stream)
                _lib.tv_pages_compact(s.shape, s.L, s.refs, *s.layers(), s.remap, s.n_live, s.ws, s.status,
                                      stream)
            stream.synchronize()
        except Exception as e:   # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in pools]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for s in pools:
        pages.fork(s.o, P, list(range(8)))
        pages.reserve(s.o, P, [8] * 8)
        code, remap, n = pages.compact(s.o, P)
        s.check([])
        assert s.n_live.tolist() == [n]


@pytest.mark.parametrize("d,dtype,comp,P", [(72, "f32", (4, 128), 1536), (512, "bf16", (4,), 512),
                                            (24, "f32", (128,), 512), (8, "bf16", (128,), 1024)])
@pytest.mark.parametrize("n_pool", [60, 8300])
def test_compact_of_other_pools(d, dtype, comp, P, n_pool):
    # fp32 rows, one compressor, both plan variants
    if n_pool > 1000:
        d = 8
    rng = np.random.default_rng(d + P)
    L = [int(x) for x in rng.integers(0, 4 * P + 1, size=12)]
    table = _random_table(rng, 12, 5, n_pool, L, P)
    for g in range(min(L[3], L[2]) // P):
        table[3][g] = table[2][g]
    extra = [p for p in (n_pool - 1, n_pool - 4, 7)]
    s = Pool(table, L, n_pool, P, d, dtype, comp, extra=extra)
    assert s.compact() == 0
    s.check([])
    assert s.compact() == 0
    s.check([])


def test_draft_steps_on_a_managed_pool():
    # the draft side's call reserves its own pages, commits nothing, and computes what it does on a
    # contiguous cache
    base = workloads.draft_beam(B=4, steps=3, L=(1500, 2600))
    for step in (1, 2, 3):
        wl = workloads.draft_level(base, step)
        wl.L[0] = 1536                    # its next position lies on a page that is not there yet
        shape, st = engine.alloc_pool(wl, 512, 40)
        rb = engine.alloc_round(wl, shape)
        engine.prefill(shape, st, rb)
        torch.cuda.synchronize()
        L, mapped = st.L.clone(), st.page_table.clone()
        engine.draft_decode(shape, st, rb)
        cshape = engine.shape_for(wl)
        cshape.raw_cap, cshape.c4_cap, cshape.c128_cap = shape.raw_cap, shape.c4_cap, shape.c128_cap
        view = st.page_table.long().clamp(min=0)
        logical = lambda t: t[view].reshape(wl.B, -1, wl.d).contiguous()
        cst = engine.DeviceState(*(logical(getattr(st, k)) for m in MS for k in MS[m]), L=L.clone())
        crb = engine.alloc_round(wl, cshape)
        engine.draft_decode(cshape, cst, crb)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == int(crb.status.item()) == 0
        for name in ("O", "lse", "scrK4", "scrV128"):
            assert torch.equal(getattr(rb, name), getattr(crb, name)), name
        assert torch.equal(st.L, L)
        new = (mapped == -1) & (st.page_table >= 0)
        assert int(new[0].sum()) == 1 and torch.equal(st.page_table[~new], mapped[~new])
        held = st.page_table[st.page_table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=40).int(), st.page_refs)
