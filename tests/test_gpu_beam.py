"""tv_beam_select on the GPU against the oracle, and beams over a managed pool.

Scores: ln S is summed in fp32 (2^-21 relative for the sums, 2^-22 for the exponentials) and stored as
the log probability of the largest logit (2^-24 of it, below 2^5), the rest is exact in fp64, the result
is rounded to fp32: 2^-20 + 2^-24 |score|.  Candidates of different beams closer than twice that could
change places; the inputs keep them 2^-12 apart unless they are equal by construction.
"""

import math

import numpy as np
import pytest
import torch

from oracle import beam
from tree_speculative_verify_gb300 import _lib, engine, workloads

pytestmark = pytest.mark.gpu


def _run(logits, scores, done, width, eos, scale, in_place=False, use_done=True, stream=None):
    B = len(scores)
    shape = _lib.make_shape(B=B, D=1, H=1, d=8, comp_mask=1)
    i = lambda: torch.full((B,), -7, dtype=torch.int32, device="cuda")
    s = torch.tensor(scores, dtype=torch.float32).cuda()
    d = torch.tensor(done, dtype=torch.int32).cuda() if use_done else None
    out = dict(source=i(), token=i(), new_scores=s if in_place else torch.full_like(s, 5.0),
               new_done=d if in_place and use_done else i(), rank=i())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((_lib.tv_beam_workspace_size(shape, width),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _lib.tv_beam_select(shape, width, logits, s, d, eos, scale, out["source"], out["token"],
                        out["new_scores"], out["new_done"], out["rank"], ws, status, stream)
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in out.items()}, status.item()


def _check(logits, scores, done, width, eos, scale, **kw):
    got, status = _run(logits, scores, done, width, eos, scale, **kw)
    x = logits.double().cpu().numpy()
    codes = []
    for g in range(len(scores) // width):
        at = slice(g * width, g * width + width)
        code, rows = beam.select_group(x[at], np.float32(scores)[at], done[at], eos, scale)
        codes.append(code)
        for w, (source, token, score, ended, rank) in enumerate(rows):
            b = g * width + w
            want = (source + g * width if source >= 0 else -1, token, ended, rank)
            assert (got["source"][b], got["token"][b], got["new_done"][b], got["rank"][b]) == want, b
            if math.isinf(score):
                assert got["new_scores"][b] == score
            else:
                assert abs(got["new_scores"][b] - score) <= 2.0 ** -20 + 2.0 ** -24 * abs(score)
    assert status == min(codes)
    return got


def _apart(logits, scores, done, width, scale):
    """Whether a group's candidates near the chosen ones are equal or at least 2^-12 apart."""
    for g in range(len(scores) // width):
        found = []
        for b in range(g * width, g * width + width):
            if done[b]:
                found.append(scores[b])
            elif scores[b] > -math.inf:
                lp = torch.log_softmax(logits[b].double() * scale, 0)
                found += [float(np.float32(scores[b])) + v for v in set(torch.topk(lp, min(width + 1, len(lp)))[0].tolist())]
        found = sorted(f for f in found if f > -math.inf)[-(width + 1):]
        if any(0 < b - a < 2.0 ** -12 for a, b in zip(found, found[1:])):
            return False
    return True


def _case(G, width, V, dtype, seed, pad=0, masked=False, ended=0.0, first=False, scale=1.0):
    """Inputs whose candidates keep their distance: the first such seed."""
    for k in range(200):
        g = torch.Generator().manual_seed(1000 * seed + k)
        B = G * width
        x = (2.5 * torch.randn((B, V + pad), generator=g)).to(dtype)
        x.scatter_add_(1, torch.randint(0, V, (B, 5), generator=g),
                       (4 + 8 * torch.rand((B, 5), generator=g)).to(dtype))
        if masked:
            x[::2, torch.arange(V) % 7 != 3] = -math.inf
            x[B - 1] = -math.inf
        scores = (-6 * torch.rand(B, generator=g)).tolist()
        if first:
            scores = [s if b % width == 0 else -math.inf for b, s in enumerate(scores)]
        done = (torch.rand(B, generator=g) < ended).int().tolist()
        if _apart(x[:, :V], scores, done, width, scale):
            return x.cuda()[:, :V], scores, done
    raise AssertionError("no such seed")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,width,V,pad", [(1, 1, 1, 0), (1, 4, 32000, 0), (3, 2, 1000, 1), (5, 8, 257, 3),
                                           (2, 32, 5000, 0), (1, 16, 60000, 2), (4, 3, 2, 0), (2, 7, 130001, 0)])
def test_selection_matches_the_oracle(G, width, V, pad, dtype):
    x, scores, done = _case(G, width, V, dtype, G + width, pad, ended=0.2)
    _check(x, scores, done, width, 2 % V, 1.0)


@pytest.mark.parametrize("kw", [dict(masked=True), dict(first=True), dict(ended=1.0), dict(scale=0.25),
                                dict(masked=True, ended=0.4, scale=2.0)])
def test_masks_first_steps_and_ended_beams(kw):
    x, scores, done = _case(4, 6, 500, torch.bfloat16, 3, **kw)
    _check(x, scores, done, 6, 3, kw.get("scale", 1.0))


def test_ties_go_to_the_lower_beam_then_the_lower_id():
    V, width = 100, 4
    x = torch.zeros((8, V), dtype=torch.bfloat16)
    x[4:, 90:] = 1.0
    got = _check(x.cuda(), [-1.0] * 8, [0] * 8, width, 99, 1.0)
    assert got["source"][:4] == [0, 0, 0, 0] and got["token"][:4] == [0, 1, 2, 3]
    assert got["token"][4:] == [90, 91, 92, 93]


def test_few_candidates_leave_slots_without_a_source():
    x = torch.full((4, 50), -math.inf)
    x[2, 7] = 1.0
    got = _check(x.cuda(), [-1.0, -2.0, -3.0, -math.inf], [0, 0, 0, 0], 4, 7, 1.0)
    assert got["source"] == [-1, -1, 2, -1] and got["new_done"] == [0, 0, 1, 0]


def test_bad_values_take_their_beam_out():
    for value, scores in ((math.nan, [0.0] * 4), (math.inf, [0.0] * 4), (0.0, [0.0, math.nan, 0.5, math.inf])):
        g = torch.Generator().manual_seed(4)
        x = torch.randn((4, 300), generator=g)
        x[1, 200] = value
        _check(x.cuda(), scores, [0, 0, 0, 0], 4, 1, 1.0)
    x[1, 200] = math.nan      # of an ended beam or an empty slot they do not count
    _check(x.cuda(), [-0.5, -0.25, -1.0, -1.5], [0, 1, 0, 0], 4, 1, 1.0)
    _check(x.cuda(), [-0.5, -math.inf, -1.0, -1.5], [0, 0, 0, 0], 4, 1, 1.0)


def test_in_place_without_done_and_on_another_stream():
    x, scores, done = _case(6, 5, 3001, torch.float32, 5)
    _check(x, scores, done, 5, 2, 1.0, in_place=True)
    _check(x, scores, [0] * 30, 5, 2, 1.0, use_done=False)
    other = torch.cuda.Stream()
    _check(x, scores, done, 5, 2, 1.0, stream=other)


def test_captured_steps_replay():
    x, scores, done = _case(8, 4, 4000, torch.bfloat16, 6)
    B = 32
    shape = _lib.make_shape(B=B, D=1, H=1, d=8, comp_mask=1)
    s0 = torch.tensor(scores, dtype=torch.float32).cuda()
    i = lambda: torch.zeros(B, dtype=torch.int32, device="cuda")
    s, d, source, token, rank, status = s0.clone(), i(), i(), i(), i(), i()
    ws = torch.empty(_lib.tv_beam_workspace_size(shape, 4), dtype=torch.uint8, device="cuda")

    def step():
        _lib.tv_beam_select(shape, 4, x, s, d, 2, 1.0, source, token, s, d, rank, ws, status)

    def twice(go):
        s.copy_(s0)
        d.zero_()
        go(), go()
        torch.cuda.synchronize()
        return [t.clone() for t in (s, d, source, token, rank)]

    want = twice(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert all(torch.equal(a, b) for a, b in zip(twice(graph.replay), want))
    assert status[0].item() == 0


def _two_groups(n_pool_pages):
    """Two groups of two beams, their first steps ahead: one request of 100 tokens, one of 50."""
    wl = workloads.make_workload("beams", B=4, D=1, H=2, d=64, W=8, tail_mode="window", ms=(4, 128), dtype="f32",
                                 L=[100, 0, 50, 0], k=1, steps=1, p_match=0.5, seed=3, kv_scale=0.5)
    shape, st = engine.alloc_pool(wl, page_tokens=512, n_pool_pages=n_pool_pages)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    return shape, st, rb, engine.alloc_beams(shape, width=2, eos=5)


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_step_that_runs_out_of_pages_can_be_repeated(own_stream):
    """The copies of both groups' partial pages need two pages more than the two that are held.  The failed
    step is taken back, one group given up, and the step repeated as it goes in a pool with room."""
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((4, 40), generator=g).cuda()
    want_shape, want_st, want_rb, want = _two_groups(8)
    engine.beam_step(want_shape, want_st, want_rb, want, logits)
    shape, st, rb, beams = _two_groups(2)
    stream = torch.cuda.Stream() if own_stream else None
    before = [t.clone() for t in (beams.scores, beams.done, st.L, st.page_table, st.page_refs)]
    torch.cuda.synchronize()
    engine.beam_step(shape, st, rb, beams, logits, stream=stream)
    torch.cuda.synchronize()
    assert rb.status.item() == -4 and not torch.equal(beams.scores, before[0])
    assert all(torch.equal(a, b) for a, b in zip((st.L, st.page_table, st.page_refs), before[2:]))
    engine.beam_undo(beams, stream)
    torch.cuda.synchronize()
    assert torch.equal(beams.scores, before[0]) and torch.equal(beams.done, before[1])
    rb.status.zero_()
    beams.scores[2:] = -math.inf
    torch.cuda.synchronize()
    engine.beam_step(shape, st, rb, beams, logits, stream=stream)
    torch.cuda.synchronize()
    assert rb.status.item() == 0 and want_rb.status.item() == 0
    for a, b in ((beams.scores, want.scores), (beams.token, want.token), (beams.source, want.source),
                 (st.L, want_st.L)):
        assert torch.equal(a[:2], b[:2])
    assert beams.source[2:].tolist() == [-1, -1] and st.L.tolist() == [100, 100, 0, 0]
    for b in range(2):
        for name, m in (("rawK", 1), ("rawV", 1), ("c4K", 4), ("c4V", 4)):
            rows = [getattr(x, name)[int(x.page_table[b, 0])][:100 // m] for x in (st, want_st)]
            assert torch.equal(*rows), name


def test_captured_steps_keep_what_is_in_front_of_the_last():
    """A captured step, replayed twice: undoing takes back the second replay."""
    shape, st, rb, beams = _two_groups(12)
    x = torch.randn((4, 40), generator=torch.Generator().manual_seed(6)).cuda()
    engine.beam_step(shape, st, rb, beams, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        engine.beam_step(shape, st, rb, beams, x, stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    scores, done = beams.scores.clone(), beams.done.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert rb.status.item() == 0 and not torch.equal(beams.scores, scores)
    engine.beam_undo(beams)
    assert torch.equal(beams.scores, scores) and torch.equal(beams.done, done)


def test_beams_over_a_managed_pool():
    """Beam search over a toy model whose keys, values and logits depend on the whole sequence: a prompt
    in one chunk, then beams that are selected, reordered and extended.  The pool's beams must hold the
    caches of the sequences that a plain search over token lists keeps."""
    G, width, d, H, V, eos, steps = 2, 3, 64, 2, 40, 5, 9
    prompts = [[7, 3, 9] * 45, [1, 8]]
    B = G * width
    g = torch.Generator().manual_seed(8)
    emb = torch.randn((V, 3, d), generator=g).cuda()
    head = (0.7 * torch.randn((H * d, V), generator=g)).cuda()
    wl = workloads.make_workload("beams", B=B, D=1, H=H, d=d, W=8, tail_mode="window", ms=(4, 128),
                                 dtype="f32", L=[0] * B, k=1, steps=1, p_match=0.5, seed=1, kv_scale=0.5)
    wl.raw_cap = 512
    wl.rawK = wl.rawV = torch.zeros((B, 512, d))
    shape, st = engine.alloc_pool(wl, page_tokens=512, n_pool_pages=2 * B + 2)
    rb = engine.alloc_round(wl, shape)
    f = (50.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()

    def forward(news):
        """Appends news[b] tokens to every slot; the logits of the last one of each."""
        flat = [t for n in news for t in n]
        starts = torch.tensor(np.cumsum([0] + [len(n) for n in news]), dtype=torch.int32).cuda()
        x = emb[torch.tensor(flat).cuda()]
        need = torch.tensor([len(n) for n in news], dtype=torch.int32).cuda()
        engine.reserve(shape, st, rb, need)
        Q = x[:, 2, None].expand(-1, H, d).contiguous()
        engine.append(shape, st, rb, starts, x[:, 0].contiguous(), x[:, 1].contiguous(), Q, d, 1, f)
        O, _ = engine.chunk_attention(shape, st, rb, starts, Q, engine.alloc_chunk(shape, len(flat)))
        out = torch.zeros((B, V), device="cuda")
        for b, n in enumerate(news):
            if n:
                out[b] = O[int(starts[b + 1]) - 1].reshape(-1) @ head
        torch.cuda.synchronize()
        assert rb.status.item() == 0
        return out

    def logits_of(sequence):
        """The same model on one sequence from scratch, in a pool of its own: its last token's logits."""
        sh, s1 = engine.alloc_pool(one, page_tokens=512, n_pool_pages=2)
        engine.reserve(sh, s1, rb1, torch.tensor([len(sequence)], dtype=torch.int32).cuda())
        x = emb[torch.tensor(sequence).cuda()]
        starts = torch.tensor([0, len(sequence)], dtype=torch.int32).cuda()
        Q = x[:, 2, None].expand(-1, H, d).contiguous()
        engine.append(sh, s1, rb1, starts, x[:, 0].contiguous(), x[:, 1].contiguous(), Q, d, 1, f)
        O, _ = engine.chunk_attention(sh, s1, rb1, starts, Q, engine.alloc_chunk(sh, len(sequence)))
        return O[-1].reshape(-1) @ head

    one = workloads.make_workload("one", B=1, D=1, H=H, d=d, W=8, tail_mode="window", ms=(4, 128),
                                  dtype="f32", L=[0], k=1, steps=1, p_match=0.5, seed=1, kv_scale=0.5)
    one.raw_cap, one.g = 512, wl.g
    one.rawK = one.rawV = torch.zeros((1, 512, d))
    rb1 = engine.alloc_round(one, engine.alloc_pool(one, page_tokens=512, n_pool_pages=2)[0])

    beams = engine.alloc_beams(shape, width, eos)
    texts = [prompts[b // width] if b % width == 0 else None for b in range(B)]
    logits = forward([t or [] for t in texts])
    for step in range(steps):
        scores, done = beams.scores.tolist(), beams.done.tolist()
        engine.beam_step(shape, st, rb, beams, logits)
        torch.cuda.synchronize()
        assert rb.status.item() == 0
        x = logits.double().cpu().numpy()
        source, token = beams.source.tolist(), beams.token.tolist()
        for q in range(G):
            at = slice(q * width, q * width + width)
            rows = beam.select_group(x[at], scores[at], done[at], eos, 1.0)[1]
            assert [r[1] for r in rows] == token[at]
            assert [r[0] + q * width if r[0] >= 0 else -1 for r in rows] == source[at]
        ended = [s >= 0 and done[s] for s in source]
        texts = [None if s < 0 else texts[s] + ([] if e else [t])
                 for s, t, e in zip(source, token, ended)]
        logits = forward([[t] if s >= 0 and not e else [] for s, t, e in zip(source, token, ended)])
        assert st.L.tolist() == [0 if t is None else len(t) for t in texts]
        for b in (step % B, (step + 4) % B):
            if texts[b] is not None and not ended[b]:
                # the same sums in another order: fp32, values of a few units
                assert (logits_of(texts[b]) - logits[b]).abs().max() <= 1e-3
    assert max(len(t) for t in texts if t) > 130
